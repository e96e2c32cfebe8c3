// lora.cu -- low-rank adapters of many requests beside a shared projection:
//     V[m,r]  = s_a sum_k X[m,k] A[a][r][k]                 a = adapters[m], r < r_a
//     Y[m,n]  = base[m,n] + sum_{r < r_a} V[m,r] B[a][n][r]  base = X W^T (skinny_gemm_bf16)
// Three launches: the first (shrink) writes V in fp32, the second is the
// projection, the third (expand) adds.  Both adapter kernels are bound by the
// bytes of A and B, read once per adapter that occurs: the CTAs of the first
// token of an adapter (its leader) serve every token that shares it, the CTAs
// of the others leave.
//
// With programmatic dependent launch the shrink kernel lets the projection
// start only after its own wait: what was launched before this call is then
// complete for all three kernels, so the expand kernel may read the adapters'
// ids and B before it waits for the projection.
#include "dotload.cuh"
#include "experts_gemm.h"

namespace skinny {
namespace {

constexpr int kMaxM = SKINNY_MAX_M;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 8;              // tokens held at a time

// The tokens that share token m's adapter, if m is the first of them: their
// number, 0 otherwise.  Tokens without an adapter count as sharing one.  list:
// kMaxM ints.  Every thread of the CTA takes part.
__device__ __forceinline__ int adapter_group(const int32_t *adapters, int M, int L, int m, int *list, int *adapter) {
    __shared__ int s_id[kMaxM];
    __shared__ int s_count;
    for (int i = threadIdx.x; i < M; i += blockDim.x) {
        const int id = __ldcg(adapters + i);
        s_id[i] = (unsigned)id < (unsigned)L ? id : -1;
    }
    __syncthreads();
    const int a = s_id[m];
    if (threadIdx.x < 32) {
        int n = 0;
        bool first = true;
        for (int i0 = 0; i0 < M; i0 += 32) {
            const int i = i0 + threadIdx.x;
            const unsigned same = __ballot_sync(0xFFFFFFFFu, i < M && s_id[i] == a);
            if (same && i0 + __ffs(same) - 1 < m) first = false;
            if (same >> threadIdx.x & 1) list[n + __popc(same & ((1u << threadIdx.x) - 1))] = i;
            n += __popc(same);
        }
        if (threadIdx.x == 0) s_count = first ? n : 0;
    }
    __syncthreads();
    *adapter = a;
    return s_count;
}

__device__ __forceinline__ int adapter_rank(const int32_t *ranks, int a, int R) {
    return ranks ? max(0, min(R, __ldcg(ranks + a))) : R;
}

// Grid (ceil(R / 2), M).  Two rows of A per CTA, four warps along K each: warp
// q takes the 256-element pieces q, q + 4, ... of its row against eight tokens
// at a time, and the four sums are added in order.
constexpr int kShrinkRows = 2;
constexpr int kShrinkParts = kWarps / kShrinkRows;
template <int V>
__global__ void __launch_bounds__(kThreads)
lora_shrink_kernel(const uint16_t *__restrict__ X, int64_t ldx, const uint16_t *__restrict__ A, int64_t lda,
                   int64_t ldae, const int32_t *__restrict__ adapters, const int32_t *__restrict__ ranks,
                   const float *__restrict__ scales, int L, int R, int M, int K, float *__restrict__ Vout)
{
    __shared__ int list[kMaxM];
    __shared__ float part[kShrinkRows][kShrinkParts][kTile];
    griddep_wait();
    griddep_launch_dependents();
    int a;
    const int count = adapter_group(adapters, M, L, blockIdx.y, list, &a);
    if (count == 0 || a < 0) return;
    const int rank = adapter_rank(ranks, a, R);
    const int r0 = blockIdx.x * kShrinkRows;
    if (r0 >= rank) return;
    const float scale = scales ? __ldcg(scales + a) : 1.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = warp / kShrinkParts, q = warp % kShrinkParts;
    const bool live = r0 + row < rank;
    const uint16_t *ar = A + (int64_t)a * ldae + (int64_t)(live ? r0 + row : r0) * lda;
    for (int t0 = 0; t0 < count; t0 += kTile) {
        float acc[kTile];
#pragma unroll
        for (int t = 0; t < kTile; ++t) acc[t] = 0.f;
        if (live) {
            for (int k0 = q * 256; k0 < K; k0 += kShrinkParts * 256) {
                float w[8];
                load8<V, true>(ar, k0, K, lane, w);
#pragma unroll
                for (int t = 0; t < kTile; ++t) {
                    if (t0 + t >= count) break;
                    float x[8], p = 0.f;
                    load8<V, false>(X + (int64_t)list[t0 + t] * ldx, k0, K, lane, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) p = fmaf(w[j], x[j], p);
                    acc[t] += p;
                }
            }
        }
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            if (t0 + t >= count) break;
            acc[t] = warp_sum(acc[t]);
            if (lane == 0) part[row][q][t] = acc[t];
        }
        __syncthreads();
        const int t = threadIdx.x % kTile, rr = threadIdx.x / kTile;
        if (rr < kShrinkRows && r0 + rr < rank && t0 + t < count) {
            float s = part[rr][0][t];
            for (int i = 1; i < kShrinkParts; ++i) s += part[rr][i][t];
            Vout[(int64_t)list[t0 + t] * R + r0 + rr] = s * scale;
        }
        __syncthreads();
    }
}

// Grid (ceil(N / kExpandCols), M).  G lanes share a row of B, eight elements
// each (G = the power of two covering R / 8), so a warp holds 32 / G outputs at
// once; a lane's eight V of eight tokens stay in registers while the rows of B
// stream past.  The sums of a CTA's columns are gathered in shared memory and
// added to the base in whole rows.
constexpr int kExpandCols = 128;
template <int V>
__global__ void __launch_bounds__(kThreads)
lora_expand_kernel(const uint16_t *__restrict__ B, int64_t ldb, int64_t ldbe, const int32_t *__restrict__ adapters,
                   const int32_t *__restrict__ ranks, int L, int R, int G, int M, int N, const float *__restrict__ Vin,
                   const float *base, int64_t ldbase, void *Y, int64_t ldy, int out_bf16)
{
    __shared__ int list[kMaxM];
    __shared__ float add[kTile][kExpandCols];
    griddep_launch_dependents();
    int a;
    const int count = adapter_group(adapters, M, L, blockIdx.y, list, &a);
    const int rank = a >= 0 ? adapter_rank(ranks, a, R) : 0;
    griddep_wait();
    if (count == 0 || (a < 0 && !out_bf16)) return;   // nothing to add, and fp32: the base is Y
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n0 = blockIdx.x * kExpandCols, cols = min(kExpandCols, N - n0);
    const int c = lane % G, per = 32 / G;
    for (int t0 = 0; t0 < count; t0 += kTile) {
        const int tn = min(kTile, count - t0);
        if (rank > 0) {
            float v[kTile][8];
#pragma unroll
            for (int t = 0; t < kTile; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[t][j] = (t < tn && 8 * c + j < rank) ? __ldcg(Vin + (int64_t)list[t0 + t] * R + 8 * c + j) : 0.f;
            for (int i = warp * per + lane / G; i < kExpandCols; i += kWarps * per) {
                float b[8];
                const uint16_t *row = B + (int64_t)a * ldbe + (int64_t)(n0 + min(i, cols - 1)) * ldb + 8 * c;
                const int len = rank - 8 * c;
                // a vector never passes the row's R elements; what lies past the rank becomes 0
#pragma unroll
                for (int u = 0; u < 8; u += V) {
                    if (u + V <= len) {
                        if constexpr (V == 8) {
                            const uint4 q = ldg_stream_v4(row);
                            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int h = 0; h < 4; ++h) { b[2 * h] = bf16_lo(w[h]); b[2 * h + 1] = bf16_hi(w[h]); }
                        } else if constexpr (V == 4) {
                            const uint2 q = ldg_stream_v2(row + u);
                            b[u] = bf16_lo(q.x); b[u + 1] = bf16_hi(q.x); b[u + 2] = bf16_lo(q.y); b[u + 3] = bf16_hi(q.y);
                        } else if constexpr (V == 2) {
                            const uint32_t q = ldg_stream_u32(row + u);
                            b[u] = bf16_lo(q); b[u + 1] = bf16_hi(q);
                        } else {
                            b[u] = bf16_one(ldg_stream_u16(row + u));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < V; ++j) b[u + j] = u + j < len ? bf16_one(ldg_stream_u16(row + u + j)) : 0.f;
                    }
                }
#pragma unroll
                for (int t = 0; t < kTile; ++t) {
                    if (t >= tn) break;
                    float p = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) p = fmaf(b[j], v[t][j], p);
                    for (int o = G >> 1; o > 0; o >>= 1) p += __shfl_xor_sync(0xFFFFFFFFu, p, o);
                    if (c == 0) add[t][i] = p;
                }
            }
            __syncthreads();
        }
        for (int i = tid; i < tn * kExpandCols; i += kThreads) {
            const int t = i / kExpandCols, n = i % kExpandCols;
            if (n >= cols) continue;
            const int64_t m = list[t0 + t];
            const float y = __ldcg(base + m * ldbase + n0 + n) + (rank > 0 ? add[t][n] : 0.f);
            store_y(Y, out_bf16, m * ldy + n0 + n, y);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs &a, const CallCtx &c, cudaStream_t stream) {
    const uint16_t *X = a.X, *A = a.A;
    int64_t ldx = a.ldx, lda = a.lda, ldae = a.ldae;
    const int32_t *ad = a.adapters, *rk = a.ranks;
    const float *sc = a.scales;
    int L = a.L, R = a.R, M = a.M, K = a.K;
    float *V = a.V;
    void *args[] = {&X, &ldx, &A, &lda, &ldae, &ad, &rk, &sc, &L, &R, &M, &K, &V};
    const uintptr_t all = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(A) | (uintptr_t)(2 * ldx) |
                          (uintptr_t)(2 * lda) | (uintptr_t)(2 * ldae);
    const void *fn;
    switch (bf16_vec(all)) {
        case 8: fn = (const void *)lora_shrink_kernel<8>; break;
        case 4: fn = (const void *)lora_shrink_kernel<4>; break;
        case 2: fn = (const void *)lora_shrink_kernel<2>; break;
        default: fn = (const void *)lora_shrink_kernel<1>; break;
    }
    return launch_plain(fn, dim3((R + kShrinkRows - 1) / kShrinkRows, M), kThreads, 0, stream, c.pdl, args);
}

cudaError_t launch_lora_expand(const LoraArgs &a, const CallCtx &c, cudaStream_t stream) {
    const uint16_t *B = a.B;
    int64_t ldb = a.ldb, ldbe = a.ldbe, ldbase = a.ldbase, ldy = a.ldy;
    const int32_t *ad = a.adapters, *rk = a.ranks;
    int L = a.L, R = a.R, M = a.M, N = a.N, ob = a.out_bf16, G = 1;
    while (8 * G < R) G *= 2;
    const float *V = a.V, *base = a.base;
    void *Y = a.Y;
    void *args[] = {&B, &ldb, &ldbe, &ad, &rk, &L, &R, &G, &M, &N, &V, &base, &ldbase, &Y, &ldy, &ob};
    const uintptr_t all = reinterpret_cast<uintptr_t>(B) | (uintptr_t)(2 * ldb) | (uintptr_t)(2 * ldbe);
    const void *fn;
    switch (bf16_vec(all)) {
        case 8: fn = (const void *)lora_expand_kernel<8>; break;
        case 4: fn = (const void *)lora_expand_kernel<4>; break;
        case 2: fn = (const void *)lora_expand_kernel<2>; break;
        default: fn = (const void *)lora_expand_kernel<1>; break;
    }
    return launch_plain(fn, dim3((N + kExpandCols - 1) / kExpandCols, M), kThreads, 0, stream, c.pdl, args);
}

}  // namespace skinny
