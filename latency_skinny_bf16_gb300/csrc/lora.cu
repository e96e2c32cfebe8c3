// lora.cu -- low-rank adapters of many requests beside a shared projection:
//     V[m,r]  = s_a sum_k X[m,k] A[a][r][k]                 a = adapters[m], r < r_a
//     Y[m,n]  = base[m,n] + sum_{r < r_a} V[m,r] B[a][n][r]  base = X W^T (skinny_gemm_bf16)
// Three launches: the projection, the first product (shrink: V), the second
// (expand: added to the projection).  V keeps the 24 bits of fp32 as three bf16
// terms, operands of the expand kernel's MMAs as they stand, with zeros from an
// adapter's rank on.
// Both adapter kernels are bound by the bytes of A and B, read once per adapter
// that occurs and eight (shrink: 16) of its tokens; they take them straight from
// device memory into mma.sync operands, 16 rows at a time, at any alignment
// (mma_rows.cuh).
//
// With programmatic dependent launch the shrink kernel runs beside the
// projection.  The projection itself is launched without it, so all that
// precedes this call is complete when the shrink kernel starts: it may read X
// and write V at once, and waits for the projection only at its end.  The
// expand kernel, which waits for the shrink kernel, then follows both; before
// that it may read the adapters' ids, ranks and B.  (The shrink kernel first,
// then the projection with it: one token, 2112 x 7168, 17 us where this takes
// 10.8; 64 tokens, 24576 x 1536, where the projection leaves the SMs no room,
// 56.7 and 57.3.)
#include "experts_gemm.h"
#include "mma_rows.cuh"

namespace skinny {
namespace {

constexpr int kMaxM = SKINNY_MAX_M;

__device__ __forceinline__ int adapter_rank(const int32_t *ranks, int a, int R) {
    return ranks ? max(0, min(R, __ldcg(ranks + a))) : R;
}
__device__ __forceinline__ int adapter_id(const int32_t *adapters, int m, int L) {
    const int id = __ldcg(adapters + m);
    return (unsigned)id < (unsigned)L ? id : -1;
}

// ------------------------------------------------------------------ shrink
// Grid (RP / 16, M, S): the CTAs of the first token of an adapter serve every
// token that shares it, those of the others leave.  Sixteen rows of A per
// cluster of S CTAs, whose warps split K in pieces of 64; a CTA adds its warps'
// sums in order, the first CTA of the cluster the CTAs' (distributed shared
// memory): one CTA alone reads its rows at the rate of one SM.
constexpr int kShrinkWarps = 16;
constexpr int kShrinkTT = 2;           // tokens per pass: 8 * 2
constexpr int kShrinkMaxCluster = 8;

struct ShrinkParams {
    const uint16_t *X;
    int64_t ldx;
    const uint16_t *A;
    int64_t lda, ldae;
    const int32_t *adapters, *ranks;
    const float *scales;
    int L, R, M, K;
    uint16_t *V;         // [M][3][RP], RP = lora_padded_rank(R)
    int S;               // CTAs of a cluster along K
    Extent xe, ae;
};

// The three terms of v, each the top 8 bits of what the terms before it leave,
// so that they hold all 24 of v and share its sign.  A term that would be zero
// beside a v that is not becomes 2^-126 of that sign: an infinite element of B
// then meets no zero, and its products with the terms add up to what its product
// with v is.  (That adds at most 2^-125 of an element of B.)
__device__ __forceinline__ void split3(float v, uint16_t &h, uint16_t &m, uint16_t &l) {
    const uint32_t bits = __float_as_uint(v), tiny = (bits >> 16 & 0x8000u) | 0x0080u;
    const float r = isfinite(v) ? v - __uint_as_float(bits & 0xFFFF0000u) : 0.f;
    const uint32_t mb = __float_as_uint(r) >> 16;
    const uint32_t lb = __float_as_uint(r - __uint_as_float(mb << 16)) >> 16;
    h = isnan(v) ? 0x7FFF : (uint16_t)(bits >> 16);
    m = (uint16_t)(v != 0.f && (mb & 0x7FFFu) == 0 ? tiny : mb);
    l = (uint16_t)(v != 0.f && (lb & 0x7FFFu) == 0 ? tiny : lb);
}

template <bool ALIGNED>
__device__ __forceinline__ void lora_shrink(const ShrinkParams &p)
{
    __shared__ int s_id[kMaxM], list[kMaxM];
    __shared__ int s_count;
    __shared__ __align__(16) float part[kShrinkWarps][kShrinkTT][32][4];
    __shared__ float sums[kShrinkMaxCluster][kShrinkTT * 128];      // of the cluster's CTAs, in the first one
    const int S = p.S, rank_k = S > 1 ? (int)cluster_ctarank() : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int m = blockIdx.y, M = p.M, R = p.R, K = p.K;
    const int a = adapter_id(p.adapters, m, p.L);
    if (a < 0) return;
    const int rank = adapter_rank(p.ranks, a, R);
    const float scale = p.scales ? __ldcg(p.scales + a) : 1.f;
    if (tid < M) s_id[tid] = adapter_id(p.adapters, tid, p.L);
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        bool first = true;
        for (int i0 = 0; i0 < M; i0 += 32) {
            const int i = i0 + lane;
            const unsigned same = __ballot_sync(0xFFFFFFFFu, i < M && s_id[i] == a);
            if (same && i0 + __ffs(same) - 1 < m) first = false;
            if (same >> lane & 1) list[n + __popc(same & ((1u << lane) - 1))] = i;
            n += __popc(same);
        }
        if (lane == 0) s_count = first ? n : 0;
    }
    __syncthreads();
    const int count = s_count;
    const int r0 = blockIdx.x * 16;
    if (count == 0) return;
    const int RP = lora_padded_rank(R);
    if (r0 >= rank) {                  // rows past the rank: zeros
        for (int o = rank_k * 32 * kShrinkWarps + tid; o < count * 48; o += S * 32 * kShrinkWarps)
            p.V[((int64_t)list[o / 48] * 3 + o % 48 / 16) * RP + r0 + o % 16] = 0;
        return;
    }
    if (S > 1) cluster_arrive_relaxed();               // this CTA runs: its shared memory may be written
    // rows past the rank repeat its last one; their sums are not stored
    const uint16_t *Aa = p.A + (int64_t)a * p.ldae;
    const uint16_t *al = Aa + (int64_t)min(r0 + g, rank - 1) * p.lda, *ah = Aa + (int64_t)min(r0 + 8 + g, rank - 1) * p.lda;
    const int k0 = 64 * (rank_k * kShrinkWarps + warp), kstep = 64 * kShrinkWarps * S;
    for (int t0 = 0; t0 < count; t0 += 8 * kShrinkTT) {
        const int nt = min(kShrinkTT, (count - t0 + 7) / 8);
        const uint16_t *x[kShrinkTT];
        bool live[kShrinkTT];
        float acc[kShrinkTT][4];
#pragma unroll
        for (int q = 0; q < kShrinkTT; ++q) {
            live[q] = t0 + 8 * q + g < count;
            x[q] = p.X + (int64_t)list[live[q] ? t0 + 8 * q + g : t0] * p.ldx;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[q][j] = 0.f;
        }
        auto step = [&](int k, int n) {
            uint4 l[2], h[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                l[s] = load_row8<ALIGNED, true>(al, k + 32 * s + 8 * t, K, p.ae);
                h[s] = load_row8<ALIGNED, true>(ah, k + 32 * s + 8 * t, K, p.ae);
            }
#pragma unroll
            for (int q = 0; q < kShrinkTT; ++q) {
                if (q >= n) break;
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    mma_rows32(d, l[s], h[s],
                               live[q] ? load_row8<ALIGNED, false>(x[q], k + 32 * s + 8 * t, K, p.xe) : make_uint4(0, 0, 0, 0));
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[q][j] += d[j];
            }
        };
        if (nt == 1) {                 // the usual case: more steps of K in flight
#pragma unroll 4
            for (int k = k0; k < K; k += kstep) step(k, 1);
        } else {
            for (int k = k0; k < K; k += kstep) step(k, nt);
        }
#pragma unroll
        for (int q = 0; q < kShrinkTT; ++q)
            if (q < nt) *reinterpret_cast<float4 *>(part[warp][q][lane]) = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
        __syncthreads();
        if (S > 1 && t0 == 0) cluster_wait();
        const uint32_t slot = smem_u32(&sums[rank_k][0]);
        const uint32_t first = S > 1 ? mapa_shared(slot, 0) : slot;
        for (int o = tid; o < nt * 128; o += 32 * kShrinkWarps) {
            const int q = o >> 7, sl = (o >> 2) & 31, j = o & 3;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kShrinkWarps; ++w) s += part[w][q][sl][j];
            st_shared_cluster_f32(first + 4 * o, s);
        }
        auto meet = [&] {
            if (S > 1) {
                cluster_arrive_release();
                cluster_wait_acquire();
            } else {
                __syncthreads();
            }
        };
        meet();
        if (rank_k == 0) {
            for (int o = tid; o < nt * 128; o += 32 * kShrinkWarps) {
                const int q = o >> 7, sl = (o >> 2) & 31, j = o & 3;
                float s = sums[0][o];
                for (int w = 1; w < S; ++w) s += sums[w][o];
                const int i = t0 + 8 * q + 2 * (sl & 3) + (j & 1), r = r0 + (sl >> 2) + 8 * (j >> 1);
                if (i < count) {
                    uint16_t *v = p.V + (int64_t)list[i] * 3 * RP + r;
                    split3(r < rank ? s * scale : 0.f, v[0], v[RP], v[2 * RP]);
                }
            }
        }
        meet();                        // the sums are read before the next tokens', and before a CTA leaves
    }
}

template <bool ALIGNED>
__global__ void __launch_bounds__(32 * kShrinkWarps)
lora_shrink_kernel(const ShrinkParams p)
{
    griddep_launch_dependents();
    lora_shrink<ALIGNED>(p);
    griddep_wait();                    // the projection: what follows this kernel follows both
}

// ------------------------------------------------------------------ expand
// Persistent CTAs.  Each builds the list of adapters that occur, with their
// tokens, while the projection still runs; the line of (adapter, block of rows
// of B) is then dealt to the warps, which do not meet again.  A warp takes up
// to 4 x 16 rows of B at a time against eight tokens, 32 columns (two k16 MMA
// steps, three terms of V) at a time: at most six MMAs are summed in the
// tensor core before a rounded add.
constexpr int kExpandWarps = 8;
constexpr int kExpandTiles = 4;
constexpr int kExpandCtas = 2;         // per SM

struct ExpandParams {
    const uint16_t *B;
    int64_t ldb, ldbe;
    const int32_t *adapters, *ranks;
    int L, R, M, N;
    const uint16_t *V;
    const float *base;
    int64_t ldbase;
    void *Y;
    int64_t ldy;
    int out_bf16;
    Extent be;
};

// T x 16 rows of one adapter's B from row n0, for its tokens tok[0, cnt).  FULL: all of them below N.
template <bool ALIGNED, int T, bool FULL>
__device__ __forceinline__ void expand_piece(const ExpandParams &p, const uint16_t *Ba, int n0, int rank, int RP,
                                             const int *tok, int cnt, int g, int t) {
    const int N = p.N;
    // rows past the end repeat the last one; they are not stored
    const uint16_t *row[T][2];
    bool inside = true;
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = n0 + 16 * j + 8 * h + g;
            row[j][h] = Ba + (int64_t)(FULL ? n : min(n, N - 1)) * p.ldb + 8 * t;
            if (!ALIGNED) inside = inside && row_inside(row[j][h] - 8 * t, rank, p.be);
        }
    if (!ALIGNED) inside = __all_sync(0xFFFFFFFFu, inside);
    for (int t0 = 0; t0 < cnt; t0 += 8) {
        // the base of this lane's results, which the products are added to: rows g, g + 8 of each tile, tokens 2t, 2t + 1
        float acc[T][4];
        bool mine[2];
        int64_t m[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            mine[c] = t0 + 2 * t + c < cnt;
            m[c] = tok[mine[c] ? t0 + 2 * t + c : t0];
            const float *b = p.base + m[c] * p.ldbase + n0 + g;
#pragma unroll
            for (int j = 0; j < T; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    acc[j][2 * h + c] = 0.f;
                    if (mine[c] && (FULL || n0 + 16 * j + 8 * h + g < N)) acc[j][2 * h + c] = __ldcg(b + 16 * j + 8 * h);
                }
        }
        const bool live = t0 + g < cnt;
        const uint16_t *v = p.V + (int64_t)tok[live ? t0 + g : t0] * 3 * RP + 8 * t;
        auto terms = [&](int r, uint4 (&vt)[3]) {
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                vt[i] = make_uint4(0, 0, 0, 0);
                if (live) vt[i] = ldg_v4(v + i * RP + r);
            }
        };
        auto products = [&](int j, const uint4 &lo, const uint4 &hi, const uint4 (&vt)[3]) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_rows32(d, lo, hi, vt[2]);
            mma_rows32(d, lo, hi, vt[1]);
            mma_rows32(d, lo, hi, vt[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[j][c] += d[c];
        };
        int r = 0;
        if (inside) {
            for (; r + 64 <= rank; r += 64) {
                uint4 w[T][2][2], vt[2][3];
#pragma unroll
                for (int j = 0; j < T; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int s = 0; s < 2; ++s) w[j][h][s] = load_whole8<ALIGNED, true>(row[j][h], r + 32 * s);
                terms(r, vt[0]);
                terms(r + 32, vt[1]);
#pragma unroll
                for (int j = 0; j < T; ++j)
#pragma unroll
                    for (int s = 0; s < 2; ++s) products(j, w[j][0][s], w[j][1][s], vt[s]);
            }
            if (r + 32 <= rank) {
                uint4 w[T][2], vt[3];
#pragma unroll
                for (int j = 0; j < T; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[j][h] = load_whole8<ALIGNED, true>(row[j][h], r);
                terms(r, vt);
#pragma unroll
                for (int j = 0; j < T; ++j) products(j, w[j][0], w[j][1], vt);
                r += 32;
            }
        }
        for (; r < rank; r += 32) {    // the last columns, or rows at an end of B
            uint4 w[T][2], vt[3];
            const bool whole = inside && r + 8 * t + 8 <= rank;
#pragma unroll
            for (int j = 0; j < T; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[j][h] = make_uint4(0, 0, 0, 0);
                    if (whole) w[j][h] = load_whole8<ALIGNED, true>(row[j][h], r);
                }
            if (!whole && r + 8 * t < rank) {
#pragma unroll
                for (int j = 0; j < T; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[j][h] = load_row8<ALIGNED, true>(row[j][h], r, rank - 8 * t, p.be);
            }
            terms(r, vt);
#pragma unroll
            for (int j = 0; j < T; ++j) products(j, w[j][0], w[j][1], vt);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int64_t at = m[c] * p.ldy + n0 + g;
#pragma unroll
            for (int j = 0; j < T; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (mine[c] && (FULL || n0 + 16 * j + 8 * h + g < N))
                        store_y(p.Y, p.out_bf16, at + 16 * j + 8 * h, acc[j][2 * h + c]);
        }
    }
}

template <bool ALIGNED>
__global__ void __launch_bounds__(32 * kExpandWarps, kExpandCtas)
lora_expand_kernel(const ExpandParams p)
{
    __shared__ int s_id[kMaxM], s_lead[kMaxM], list[kMaxM];
    __shared__ int g_first[kMaxM], g_count[kMaxM], g_adapter[kMaxM], g_rank[kMaxM];
    __shared__ int s_groups;
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int M = p.M, N = p.N, R = p.R, RP = lora_padded_rank(R);
    if (tid == 0) s_groups = 0;
    if (tid < M) s_id[tid] = adapter_id(p.adapters, tid, p.L);
    __syncthreads();
    // token i: its adapter's first token, its place among the tokens that share it
    int lead = 0, among = 0, count = 0;
    const bool take = tid < M && (s_id[tid] >= 0 || p.out_bf16);   // fp32: the base is Y already
    if (tid < M) {
        lead = tid;
        for (int j = M - 1; j >= 0; --j)
            if (s_id[j] == s_id[tid]) {
                lead = j;
                ++count;
                among += j < tid ? 1 : 0;
            }
        s_lead[tid] = take ? lead : kMaxM;
    }
    __syncthreads();
    if (take) {
        int before = 0, group = 0;
        for (int j = 0; j < M; ++j) {
            before += s_lead[j] < lead ? 1 : 0;
            group += (s_lead[j] == j && j < lead) ? 1 : 0;
        }
        list[before + among] = tid;
        if (lead == tid) {
            g_first[group] = before;
            g_count[group] = count;
            g_adapter[group] = s_id[tid];
            g_rank[group] = s_id[tid] >= 0 ? adapter_rank(p.ranks, s_id[tid], R) : 0;
            atomicMax(&s_groups, group + 1);
        }
    }
    __syncthreads();
    const int groups = s_groups;
    const int warps = (int)gridDim.x * kExpandWarps;
    // rows per piece: 64, or 16 while that leaves warps without work
    const int tiles = (int64_t)groups * ((N + 16 * kExpandTiles - 1) / (16 * kExpandTiles)) < warps ? 1 : kExpandTiles;
    const int pieces = (N + 16 * tiles - 1) / (16 * tiles);
    const int64_t first = (int64_t)blockIdx.x + (int64_t)gridDim.x * warp, end = (int64_t)groups * pieces;
    if (first < end) {                 // the first piece's rows, on their way to L2
        const int gr = (int)(first / pieces), n0 = (int)(first - (int64_t)gr * pieces) * 16 * tiles;
        const int bytes = 2 * g_rank[gr];
        if (bytes > 0)
            for (int i = lane; i < 16 * tiles && n0 + i < N; i += 32) {
                const char *row = reinterpret_cast<const char *>(p.B + (int64_t)g_adapter[gr] * p.ldbe + (int64_t)(n0 + i) * p.ldb);
                for (int o = 0; o < bytes; o += 128) prefetch_l2(row + o);
            }
    }
    griddep_wait();
    for (int64_t u = first; u < end; u += warps) {
        const int gr = (int)(u / pieces), n0 = (int)(u - (int64_t)gr * pieces) * 16 * tiles;
        const uint16_t *Ba = p.B + (int64_t)max(0, g_adapter[gr]) * p.ldbe;
        const int rank = g_rank[gr], cnt = g_count[gr];
        const int *tok = list + g_first[gr];
        if (tiles == kExpandTiles && n0 + 16 * kExpandTiles <= N)
            expand_piece<ALIGNED, kExpandTiles, true>(p, Ba, n0, rank, RP, tok, cnt, g, t);
        else
            for (int j = 0; j < tiles && n0 + 16 * j < N; ++j)
                expand_piece<ALIGNED, 1, false>(p, Ba, n0 + 16 * j, rank, RP, tok, cnt, g, t);
    }
}

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs &a, const CallCtx &c, cudaStream_t stream) {
    // CTAs along K: for long K and few tokens, 512 of K each at least (GB300, one token, 16 x 7168 beside the
    // 2112 x 7168 projection: the whole call 14.6 us with one CTA, 10.2 with eight)
    const int tiles = lora_padded_rank(a.R) / 16;
    int S = 1;
    while (S < kShrinkMaxCluster && 2 * S * tiles * a.M <= 2 * c.num_sms && a.K >= 2 * S * 512) S *= 2;
    ShrinkParams p{a.X, a.ldx, a.A, a.lda, a.ldae, a.adapters, a.ranks, a.scales, a.L, a.R, a.M, a.K, a.V, S,
                   {addr(a.X), addr(a.X) + (uintptr_t)(2 * ((a.M - 1) * a.ldx + a.K))},
                   {addr(a.A), addr(a.A) + (uintptr_t)(2 * ((a.L - 1) * a.ldae + (a.R - 1) * a.lda + a.K))}};
    void *args[] = {&p};
    const bool al = (addr(a.X) | addr(a.A)) % 16 == 0 && (a.ldx | a.lda | a.ldae) % 8 == 0;
    return launch_plain(al ? (const void *)lora_shrink_kernel<true> : (const void *)lora_shrink_kernel<false>,
                        dim3(tiles, a.M, S), 32 * kShrinkWarps, 0, stream, c.pdl, args, S);
}

cudaError_t launch_lora_expand(const LoraArgs &a, const CallCtx &c, cudaStream_t stream) {
    ExpandParams p{a.B, a.ldb, a.ldbe, a.adapters, a.ranks, a.L, a.R, a.M, a.N, a.V, a.base, a.ldbase, a.Y, a.ldy,
                   a.out_bf16, {addr(a.B), addr(a.B) + (uintptr_t)(2 * ((a.L - 1) * a.ldbe + (a.N - 1) * a.ldb + a.R))}};
    void *args[] = {&p};
    const bool al = addr(a.B) % 16 == 0 && (a.ldb | a.ldbe) % 8 == 0;
    // two CTAs per SM, or a warp for every 16 rows of every token's adapter when these are fewer
    const int64_t pieces = (int64_t)a.M * ((a.N + 15) / 16), want = (pieces + kExpandWarps - 1) / kExpandWarps;
    const int most = kExpandCtas * c.num_sms;
    return launch_plain(al ? (const void *)lora_expand_kernel<true> : (const void *)lora_expand_kernel<false>,
                        dim3((unsigned)(want < most ? want : most)), 32 * kExpandWarps, 0, stream, c.pdl, args);
}

}  // namespace skinny
