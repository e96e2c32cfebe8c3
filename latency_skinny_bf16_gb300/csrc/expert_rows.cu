// expert_rows.cu -- rows to experts and back: the stable sort of the router's
// choices by expert with the copies of the tokens' rows, the weighted sum of
// the experts' rows per token, and its gradient.
//
// With f = t * k + j, id_f = ids[t][j], live when 0 <= id_f < E:
//     pos_f      = #{live f': id_f' < id_f} + #{live f' < f: id_f' = id_f}
//     Xs[pos_f]  = X[t]                                     (dispatch)
//     Y[t]       = sum_j w[t][j] Ys[pos_tj]                 (combine; w = 1: the gradient of dispatch)
//     dYs[pos_f] = w_f dY[t],  dw_f = <dY[t], Ys[pos_f]>    (the gradient of combine)
// No arithmetic to speak of: each is bound by the bytes of the rows (read or
// written once each), and at decode sizes by launch latency.
#include "common.cuh"
#include "expert_rows.h"
#include "mma_rows.cuh"

namespace skinny {
namespace {

constexpr int kRowThreads = 256;
constexpr int kSortCluster = 8;
constexpr int kBulkThreads = 64;
constexpr int kBulkBytes = 2048;       // of a row, per chunk
constexpr uint64_t kBulkDrainNs = 200ull * 1000 * 1000;

// ------------------------------------------------------------------ vectors
template <int BYTES> struct Vec;
template <> struct Vec<16> { using T = uint4; };
template <> struct Vec<8> { using T = uint2; };
template <> struct Vec<4> { using T = uint32_t; };
template <> struct Vec<2> { using T = uint16_t; };

__device__ __forceinline__ int load_id(const int32_t *ids, int64_t ldid, int k, int f, int E) {
    const int64_t at = ldid == k ? (int64_t)f : (int64_t)(f / k) * ldid + f % k;
    const int id = __ldcg(ids + at);
    return (unsigned)id < (unsigned)E ? id : -1;
}

// Exclusive prefix sum over the block of one value per thread; *total gets the
// sum.  scratch: 33 ints.  Every thread of the block takes part.
__device__ __forceinline__ int block_exclusive_scan(int v, int *scratch, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int own = lane < warps ? scratch[lane] : 0;
        int s = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += u;
        }
        scratch[lane] = s - own;
        if (lane == 31) scratch[32] = s;
    }
    __syncthreads();
    *total = scratch[32];
    return scratch[warp] + inc - v;
}

// The copies of one token's row: vectors [v0, v1) of X[t] to the rows pos[0..k).
// The row is read once and stored once per live entry.
template <int VB>
__device__ __forceinline__ void copy_row(const char *src, char *Xs, int64_t ldxs_bytes, const int *pos, int k, int v0,
                                         int v1) {
    using T = typename Vec<VB>::T;
    constexpr int U = 4;
    for (int v = v0 + (int)threadIdx.x; v < v1; v += U * kRowThreads) {
        T r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * kRowThreads < v1) r[u] = __ldcg(reinterpret_cast<const T *>(src) + v + u * kRowThreads);
        for (int j = 0; j < k; ++j) {
            const int p = pos[j];
            if (p < 0) continue;
            T *dst = reinterpret_cast<T *>(Xs + (int64_t)p * ldxs_bytes);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + u * kRowThreads < v1) dst[v + u * kRowThreads] = r[u];
        }
    }
}

// ------------------------------------------------------------------ dispatch, few entries: one launch
// Grid (T + 1, chunks).  Every CTA of a token reads all n ids (a few KB, from
// L2) and counts for its own k entries, one warp each, the entries before
// them: no CTA waits for another and there is no second launch.  The work is
// n / 32 steps a warp, so this form is kept for small n.  CTA (T, 0) counts
// the experts for the offsets.
template <int VB>
__global__ void __launch_bounds__(kRowThreads)
dispatch_small_kernel(const int32_t *__restrict__ ids, int64_t ldid, const char *__restrict__ X, int64_t ldx_bytes,
                      int T, int k, int E, int nvec, int32_t *__restrict__ pos, int32_t *__restrict__ order,
                      int32_t *__restrict__ offsets, char *__restrict__ Xs, int64_t ldxs_bytes)
{
    extern __shared__ int s_ids[];
    __shared__ int s_pos[kMaxTopk];
    __shared__ int scratch[33];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = T * k, t = blockIdx.x;
    if (t == T) {
        if (blockIdx.y) return;
        int *hist = s_ids;                          // E ints
        for (int e = tid; e < E; e += kRowThreads) hist[e] = 0;
        __syncthreads();
        for (int f = tid; f < n; f += kRowThreads) {
            const int id = load_id(ids, ldid, k, f, E);
            if (id >= 0) atomicAdd(&hist[id], 1);   // whole numbers: any order gives the same counts
        }
        __syncthreads();
        const int per = (E + kRowThreads - 1) / kRowThreads;
        int sum = 0, total = 0;
        for (int i = 0; i < per; ++i)
            if (tid * per + i < E) sum += hist[tid * per + i];
        int run = block_exclusive_scan(sum, scratch, &total);
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < E) {
                offsets[e] = run;
                run += hist[e];
            }
        }
        if (tid == 0) offsets[E] = total;
        if (order)
            for (int p = total + tid; p < n; p += kRowThreads) order[p] = -1;
        return;
    }
    for (int f = tid; f < n; f += kRowThreads) s_ids[f] = load_id(ids, ldid, k, f, E);
    __syncthreads();
    for (int j = warp; j < k; j += kRowThreads / 32) {
        const int f = t * k + j, id = s_ids[f];
        int before = 0;
        for (int i = lane; i < n; i += 32) {
            const int o = s_ids[i];
            before += (o >= 0 && (o < id || (o == id && i < f))) ? 1 : 0;
        }
        before = (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)before);
        if (lane == 0) {
            const int p = id >= 0 ? before : -1;
            s_pos[j] = p;
            if (blockIdx.y == 0) {
                pos[f] = p;
                if (order && p >= 0) order[p] = f;
            }
        }
    }
    if (nvec == 0) return;
    __syncthreads();
    const int per = (nvec + gridDim.y - 1) / gridDim.y;
    const int v0 = blockIdx.y * per, v1 = min(nvec, v0 + per);
    copy_row<VB>(X + (int64_t)t * ldx_bytes, Xs, ldxs_bytes, s_pos, k, v0, v1);
}

// ------------------------------------------------------------------ dispatch, many entries: sort, then copy
// One cluster of 8 CTAs sorts: each warp owns a run of consecutive entries, so
// counting per (CTA, warp, expert) and adding in that order keeps the sort
// stable.  Pass 1 counts (entries of the same expert among 32 lanes found by
// match_any; one lane adds for all), then counts are summed over the warps and,
// through distributed shared memory, over the CTAs, and pass 2 walks the same
// entries handing out places.  No workspace, no atomics, no second launch.
__global__ void __launch_bounds__(1024)
expert_sort_kernel(const int32_t *__restrict__ ids, int64_t ldid, int k, int n, int E, int32_t *__restrict__ pos,
                   int32_t *__restrict__ order, int32_t *__restrict__ offsets)
{
    extern __shared__ int smem[];
    __shared__ int scratch[33];
    const int W = blockDim.x >> 5;
    int *hist = smem;                  // [W][E]
    int *mine = smem + W * E;          // [E] counts of this CTA, read by the others
    int *base = mine + E;              // [E] first place of this CTA's entries
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_ctarank();
    griddep_launch_dependents();
    for (int i = tid; i < W * E; i += blockDim.x) hist[i] = 0;
    griddep_wait();
    __syncthreads();
    const int64_t seg = (((int64_t)n + kSortCluster * W - 1) / (kSortCluster * W) + 31) / 32 * 32;
    const int64_t f0 = (int64_t)(rank * W + warp) * seg;
    const int steps = f0 < n ? (int)((min((int64_t)n, f0 + seg) - f0 + 31) / 32) : 0;
    int *wh = hist + warp * E;
    constexpr int U = 8;
    int id[U];
    auto read = [&](int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t f = f0 + (int64_t)(s + u) * 32 + lane;
            id[u] = (s + u < steps && f < n) ? load_id(ids, ldid, k, (int)f, E) : -1;
        }
    };
    for (int s = 0; s < steps; s += U) {
        read(s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= steps) break;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id[u]);
            if (id[u] >= 0 && lane == __ffs(same) - 1) wh[id[u]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < W; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = run;
            run += c;
        }
        mine[e] = run;
    }
    cluster_arrive_release();          // every CTA's counts are in place
    cluster_wait_acquire();
    const int per = (E + blockDim.x - 1) / blockDim.x;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        int before = 0, all = 0;
        const uint32_t at = smem_u32(mine + e);
#pragma unroll
        for (int r = 0; r < kSortCluster; ++r) {
            uint32_t c;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(mapa_shared(at, r)) : "memory");
            if (r < rank) before += (int)c;
            all += (int)c;
        }
        base[e] = sum + before;        // less the threads before this one: added below
        if (rank == 0) offsets[e] = sum;
        sum += all;
    }
    cluster_arrive_release();          // this CTA reads the others' counts no more
    int total = 0;
    const int first = block_exclusive_scan(sum, scratch, &total);
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        base[e] += first;
        if (rank == 0) offsets[e] += first;
    }
    if (rank == 0 && tid == 0) offsets[E] = total;
    if (order)
        for (int64_t p = (int64_t)total + rank * blockDim.x + tid; p < n; p += kSortCluster * blockDim.x) order[p] = -1;
    __syncthreads();
    for (int s = 0; s < steps; s += U) {
        if (steps > U) read(s);        // else the first pass has left them
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= steps) break;
            const int64_t f = f0 + (int64_t)(s + u) * 32 + lane;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id[u]);
            const int p = id[u] >= 0 ? base[id[u]] + wh[id[u]] + __popc(same & ((1u << lane) - 1)) : -1;
            __syncwarp();
            if (id[u] >= 0 && lane == __ffs(same) - 1) wh[id[u]] += __popc(same);
            __syncwarp();
            if (f < n) {
                pos[f] = p;
                if (order && p >= 0) order[p] = (int)f;
            }
        }
    }
    cluster_wait_acquire();            // no CTA leaves while its counts may be read
}

// Grid (T, chunks): the copies of a token's row, the places read from `pos`.
template <int VB>
__global__ void __launch_bounds__(kRowThreads)
dispatch_copy_kernel(const int32_t *__restrict__ pos, const char *__restrict__ X, int64_t ldx_bytes, int k, int nvec,
                     char *__restrict__ Xs, int64_t ldxs_bytes)
{
    __shared__ int s_pos[kMaxTopk];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t = blockIdx.x;
    for (int j = threadIdx.x; j < k; j += kRowThreads) s_pos[j] = __ldcg(pos + t * k + j);
    __syncthreads();
    const int per = (nvec + gridDim.y - 1) / gridDim.y;
    const int v0 = blockIdx.y * per, v1 = min(nvec, v0 + per);
    copy_row<VB>(X + t * ldx_bytes, Xs, ldxs_bytes, s_pos, k, v0, v1);
}

// ------------------------------------------------------------------ fp32 <-> stored types
// VB bytes of a bf16 or fp32 row, as loaded (through L2: rows may have just been
// written by the preceding kernel), and as fp32.
template <int VB> struct Raw {
    uint32_t w[VB >= 4 ? VB / 4 : 1];
};
template <int VB>
__device__ __forceinline__ Raw<VB> load_raw(const char *at) {
    Raw<VB> r;
    if constexpr (VB == 16) {
        const uint4 q = ldg_v4(at);
        r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
    } else if constexpr (VB == 8) {
        const uint2 q = __ldcg(reinterpret_cast<const uint2 *>(at));
        r.w[0] = q.x; r.w[1] = q.y;
    } else if constexpr (VB == 4) {
        r.w[0] = __ldcg(reinterpret_cast<const uint32_t *>(at));
    } else {
        r.w[0] = ldg_u16(at);
    }
    return r;
}
template <int VB>
__device__ __forceinline__ Raw<VB> zero_raw() {
    Raw<VB> r;
#pragma unroll
    for (int i = 0; i < (VB >= 4 ? VB / 4 : 1); ++i) r.w[i] = 0;
    return r;
}
template <bool BF16, int VB> constexpr int raw_els() { return VB / (BF16 ? 2 : 4); }
template <bool BF16, int VB>
__device__ __forceinline__ float raw_el(const Raw<VB> &r, int i) {
    if constexpr (!BF16) return __uint_as_float(r.w[i]);
    else return (i & 1) ? bf16_hi(r.w[i >> 1]) : bf16_lo(r.w[i >> 1]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)f32_to_bf16_rn(lo) | ((uint32_t)f32_to_bf16_rn(hi) << 16);
}
// N consecutive elements from element `el` of a row, each rounded once.
template <bool BF16, int N>
__device__ __forceinline__ void store_els(char *row, int64_t el, const float (&v)[N]) {
    if constexpr (BF16) {
        char *at = row + el * 2;
        if constexpr (N == 8)
            *reinterpret_cast<uint4 *>(at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                        pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        else if constexpr (N == 4)
            *reinterpret_cast<uint2 *>(at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else if constexpr (N == 2)
            *reinterpret_cast<uint32_t *>(at) = pack_bf16(v[0], v[1]);
        else
            *reinterpret_cast<uint16_t *>(at) = f32_to_bf16_rn(v[0]);
    } else {
        char *at = row + el * 4;
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4 *>(at + 4 * i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else if constexpr (N == 2) {
            *reinterpret_cast<float2 *>(at) = make_float2(v[0], v[1]);
        } else {
            *reinterpret_cast<float *>(at) = v[0];
        }
    }
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// A token's live entries, in order, in the warp's shared memory: their places,
// weights and j.  With the dropped ones left in, their loads would be missing
// from those in flight (7596 tokens x 10 x 5856 bf16, half of them dropped: 129
// us, now 90).  The weight of a dropped entry, which may be NaN, is not kept.
struct Entries {
    int p[kMaxTopk];
    float w[kMaxTopk];
    int j[kMaxTopk];
};
__device__ __forceinline__ int live_entries(Entries &e, const int32_t *pos, const float *weights, int64_t ldw,
                                            int64_t t, int k, int rows, int lane) {
    int n = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = 32 * h + lane;
        const int p = j < k ? __ldcg(pos + t * k + j) : -1;
        const float w = j < k && weights ? __ldcg(weights + t * ldw + j) : 1.f;
        const bool live = (unsigned)p < (unsigned)rows;
        const unsigned all = __ballot_sync(0xFFFFFFFFu, live);
        if (live) {
            const int at = n + __popc(all & ((1u << lane) - 1));
            e.p[at] = p;
            e.w[at] = w;
            e.j[at] = j;
        }
        n += __popc(all);
        if (k <= 32) break;
    }
    __syncwarp();
    return n;
}
// Entries per pass: as even as passes of at most eight allow.
__device__ __forceinline__ int pass_size(int n) { return n <= 8 ? n : (n + (n + 7) / 8 - 1) / ((n + 7) / 8); }

// ------------------------------------------------------------------ combine
// A warp takes one of S pieces of a token's row: the token's places are read
// once, then U rows x IT loads are in flight per lane before they are added, in
// order of j.  What limits it is the bytes in flight: a first form with a
// thread per vector spent half its time waiting for the places (8192 tokens x 8
// x 7168 bf16: 385 us, now 153, 98% of the copy rate).
template <bool IN16, bool OUT16, int VB, int U, int IT>
__device__ __forceinline__ void combine_piece(const char *__restrict__ Ys, int64_t ldys_bytes, const Entries &e, int n,
                                              int v0, int v1, char *__restrict__ y, int lane) {
    constexpr int NE = raw_els<IN16, VB>();
    const int per = pass_size(n);
    for (int vb = v0; vb < v1; vb += 32 * IT) {
        float acc[IT][NE];
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int x = 0; x < NE; ++x) acc[i][x] = 0.f;
        for (int j0 = 0; j0 < n; j0 += per) {
            const int m = min(per, n - j0);
            Raw<VB> r[U][IT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // read whatever u: a load under a branch of the warp would wait for the one before
                const char *row = Ys + (int64_t)e.p[u < m ? j0 + u : j0] * ldys_bytes;
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int v = vb + 32 * i + lane;
                    r[u][i] = (u < m && v < v1) ? load_raw<VB>(row + (int64_t)v * VB) : zero_raw<VB>();
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u >= m) break;
                const float w = e.w[j0 + u];
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int x = 0; x < NE; ++x) acc[i][x] = fmaf(w, raw_el<IN16, VB>(r[u][i], x), acc[i][x]);
            }
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int v = vb + 32 * i + lane;
            if (v < v1) store_els<OUT16, NE>(y, (int64_t)v * NE, acc[i]);
        }
    }
}
template <bool IN16, bool OUT16, int VB>
__global__ void __launch_bounds__(128)
combine_kernel(const char *__restrict__ Ys, int64_t ldys_bytes, int rows, const int32_t *__restrict__ pos,
               const float *__restrict__ weights, int64_t ldw, int T, int k, int nvec, int S, char *__restrict__ Y,
               int64_t ldy_bytes)
{
    __shared__ Entries entries[4];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = job / S;
    if (t >= T) return;
    const int seg = (int)(job - t * S);
    Entries &e = entries[threadIdx.x >> 5];
    const int n = live_entries(e, pos, weights, ldw, t, k, rows, lane);
    const int per = (nvec + S - 1) / S;
    const int v0 = seg * per, v1 = min(nvec, v0 + per);
    char *y = Y + t * ldy_bytes;
    // few entries: more of each row at a time
    constexpr int IT = VB >= 8 ? 2 : 4;
    if (n <= 2) combine_piece<IN16, OUT16, VB, 2, 4>(Ys, ldys_bytes, e, n, v0, v1, y, lane);
    else if (n <= 4) combine_piece<IN16, OUT16, VB, 4, IT>(Ys, ldys_bytes, e, n, v0, v1, y, lane);
    else combine_piece<IN16, OUT16, VB, 8, IT>(Ys, ldys_bytes, e, n, v0, v1, y, lane);
}

// Rows that start or end off 8 bytes (bf16: off 4).  Loaded element by element
// they take a request for every 128 bytes (fp32; 64 for bf16); instead the copy
// engine brings the whole 16-byte pieces that hold a chunk of each row to shared
// memory, eight rows at a time, where elements are read at any offset.  Grid
// (chunks, T).  A token one of whose rows' pieces would reach past Ys (its
// first and last row may) is read element by element.  GB300, 3001 tokens x 6 x
// 2881: fp32 51 us element by element, 45 this way (floor 34), bf16 80 and 32
// (floor 17); chunks of 4 KB and 128 threads 46 and 36, of 1 KB 69 and 45.
template <bool IN16, bool OUT16>
__global__ void __launch_bounds__(kBulkThreads)
combine_bulk_kernel(const char *__restrict__ Ys, int64_t ldys_bytes, int rows, const int32_t *__restrict__ pos,
                    const float *__restrict__ weights, int64_t ldw, int k, int H, char *__restrict__ Y, int64_t ldy_bytes,
                    int *status, uint64_t budget_ns)
{
    constexpr int ES = IN16 ? 2 : 4, PER = kBulkBytes / ES / kBulkThreads, U = 8;
    __shared__ __align__(128) char buf[U][kBulkBytes + 16];
    __shared__ Entries e;
    __shared__ __align__(8) uint64_t bar_store;
    __shared__ int s_n;
    const uint32_t bar = smem_u32(&bar_store);
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t t = blockIdx.y;
    griddep_launch_dependents();
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbarrier_init_cluster();
    }
    griddep_wait();
    if (tid < 32) {
        const int n = live_entries(e, pos, weights, ldw, t, k, rows, lane);
        if (lane == 0) s_n = n;
    }
    __syncthreads();
    const int n = s_n;
    const int first = blockIdx.x * (kBulkBytes / ES), len = min(H - first, kBulkBytes / ES);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(Ys), hi = lo + (uintptr_t)((rows - 1) * ldys_bytes + (int64_t)H * ES);
    float acc[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) acc[x] = 0.f;
    int phase = 0;
    for (int j0 = 0; j0 < n; j0 += U) {
        const int m = min(U, n - j0);
        bool inside = true;
        uint32_t bytes = 0;
        for (int u = 0; u < m; ++u) {
            const uintptr_t a = lo + (uintptr_t)((int64_t)e.p[j0 + u] * ldys_bytes + (int64_t)first * ES);
            const uintptr_t a0 = a & ~(uintptr_t)15, a1 = (a + (uintptr_t)(len * ES) + 15) & ~(uintptr_t)15;
            inside = inside && a0 >= lo && a1 <= hi;
            bytes += (uint32_t)(a1 - a0);
        }
        if (inside) {                  // the same for every thread
            if (tid == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar, bytes);
                for (int u = 0; u < m; ++u) {
                    const uintptr_t a = lo + (uintptr_t)((int64_t)e.p[j0 + u] * ldys_bytes + (int64_t)first * ES);
                    const uintptr_t a0 = a & ~(uintptr_t)15, a1 = (a + (uintptr_t)(len * ES) + 15) & ~(uintptr_t)15;
                    bulk_copy_g2s(smem_u32(buf[u]), reinterpret_cast<const void *>(a0), (uint32_t)(a1 - a0), bar);
                }
            }
            const bool got = mbar_wait_bounded(bar, (uint32_t)(phase & 1), budget_ns);
            if (__syncthreads_or(got ? 0 : 1)) {
                if (tid == 0) {
                    report_status(status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitX);
                    // the copies land before the CTA leaves
                    if (!mbar_wait_bounded(bar, (uint32_t)(phase & 1), kBulkDrainNs))
                        report_status(status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
                }
                __syncthreads();
                return;
            }
            ++phase;
        }
        for (int u = 0; u < m; ++u) {
            const float w = e.w[j0 + u];
            const char *row = Ys + (int64_t)e.p[j0 + u] * ldys_bytes + (int64_t)first * ES;
            const char *at = buf[u] + (reinterpret_cast<uintptr_t>(row) & 15);
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                const int i = x * kBulkThreads + tid;
                if (i >= len) break;
                float v;
                if constexpr (IN16) v = bf16_one(inside ? *reinterpret_cast<const uint16_t *>(at + 2 * i) : ldg_u16(row + 2 * i));
                else v = inside ? *reinterpret_cast<const float *>(at + 4 * i) : __ldcg(reinterpret_cast<const float *>(row + 4 * i));
                acc[x] = fmaf(w, v, acc[x]);
            }
        }
        __syncthreads();               // the rows are read before the next ones land
    }
    char *y = Y + t * ldy_bytes;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
        const int i = x * kBulkThreads + tid;
        const float v[1] = {acc[x]};
        if (i < len) store_els<OUT16, 1>(y, first + i, v);
    }
}

// ------------------------------------------------------------------ gradient of combine
// S warps of a CTA share a token (8 / S tokens a CTA), eight entries at a time:
// dY[t] is read once per eight entries, each Ys row read and each dYs row
// written once; the dot products stay in registers until the end of the row,
// then one butterfly and, for S > 1, the warps' sums in order.
template <bool B16, int VB, bool DW>
__global__ void __launch_bounds__(kRowThreads, 2)
combine_grad_kernel(const char *__restrict__ dY, int64_t lddy_bytes, const char *__restrict__ Ys, int64_t ldys_bytes,
                    int rows, const int32_t *__restrict__ pos, const float *__restrict__ weights, int64_t ldw, int T,
                    int k, int nvec, int S, char *__restrict__ dYs, int64_t lddys_bytes, float *__restrict__ dw,
                    int64_t lddw)
{
    constexpr int U = 8, NE = raw_els<B16, VB>(), IT = VB == 16 ? 1 : VB == 8 ? 2 : 4;
    __shared__ float part[kRowThreads / 32][kMaxTopk];      // by entry j; 0 where dropped
    __shared__ Entries entries[kRowThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 32 / S) + warp / S;
    const int seg = warp % S;
    if (t < T) {
        Entries &e = entries[warp];
        const int n = live_entries(e, pos, weights, ldw, t, k, rows, lane), size = pass_size(n);
        if constexpr (DW) {
            for (int j = lane; j < k; j += 32) part[warp][j] = 0.f;
            __syncwarp();
        }
        const char *dy = dY + t * lddy_bytes;
        const int per = (nvec + S - 1) / S;
        const int v0 = seg * per, v1 = min(nvec, v0 + per);
        for (int j0 = 0; j0 < n; j0 += size) {
            const int m = min(size, n - j0);
            int64_t p[U];
            float w[U], dot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                p[u] = e.p[u < m ? j0 + u : j0];
                w[u] = e.w[u < m ? j0 + u : j0];
                dot[u] = 0.f;
            }
            for (int vb = v0 + lane; vb < v1; vb += 32 * IT) {
                Raw<VB> g[IT], r[U][IT];
#pragma unroll
                for (int i = 0; i < IT; ++i) g[i] = vb + 32 * i < v1 ? load_raw<VB>(dy + (int64_t)(vb + 32 * i) * VB) : zero_raw<VB>();
                if constexpr (DW) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < IT; ++i)
                            r[u][i] = (u < m && vb + 32 * i < v1)
                                          ? load_raw<VB>(Ys + p[u] * ldys_bytes + (int64_t)(vb + 32 * i) * VB)
                                          : zero_raw<VB>();
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u >= m) break;
                    char *to = dYs + p[u] * lddys_bytes;
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        if (vb + 32 * i >= v1) continue;
                        float o[NE];
#pragma unroll
                        for (int x = 0; x < NE; ++x) {
                            const float gx = raw_el<B16, VB>(g[i], x);
                            o[x] = w[u] * gx;
                            if constexpr (DW) dot[u] = fmaf(gx, raw_el<B16, VB>(r[u][i], x), dot[u]);
                        }
                        store_els<B16, NE>(to, (int64_t)(vb + 32 * i) * NE, o);
                    }
                }
            }
            if constexpr (DW) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u >= m) break;
                    const float s = warp_sum(dot[u]);
                    if (lane == 0) part[warp][e.j[j0 + u]] = s;
                }
            }
        }
    }
    if constexpr (DW) {
        __syncthreads();
        if (t < T && seg == 0)
            for (int j = lane; j < k; j += 32) {
                float s = part[warp][j];
                for (int i = 1; i < S; ++i) s += part[warp + i][j];
                dw[t * lddw + j] = s;
            }
    }
}

// ------------------------------------------------------------------ rows off 8 bytes, one to many
// out[pos_f] = G[t] (kCopy: dispatch) or w_f G[t], with dw_f = <G[t], Ys[pos_f]>
// (kScaleDot), for rows that start or end off 8 bytes, where loads and stores of
// elements would bound it.  The copy engine brings a chunk of G[t] and of its
// rows of Ys to shared memory in whole 16-byte pieces; a warp per row of out
// writes whole pieces as they lie there, each from two of the chunk's shifted,
// and single elements at the chunk's ends, where a piece belongs to other rows
// too.  Grid (T, chunks; kScaleDot: 1, the dot products stay in registers).
enum Spread : int { kCopy, kScale, kScaleDot };
constexpr int kSpreadThreads = 128;
constexpr int kSpreadBytes = 2032;     // of a row per chunk: 128 pieces wherever they start
constexpr int kSpreadPitch = 2112;     // 16 bytes before the first piece and 32 behind the last are read, not used

template <bool B16, Spread MODE>
__global__ void __launch_bounds__(kSpreadThreads)
spread_bulk_kernel(const char *__restrict__ G, int64_t ldg_bytes, int T, const char *__restrict__ Ys, int64_t ldys_bytes,
                   int rows, const int32_t *__restrict__ pos, const float *__restrict__ weights, int64_t ldw, int k, int H,
                   char *__restrict__ out, int64_t ldo_bytes, float *__restrict__ dw, int64_t lddw, int *status,
                   uint64_t budget_ns)
{
    constexpr bool DOT = MODE == kScaleDot;
    constexpr int ES = B16 ? 2 : 4, NE = 16 / ES, PER = kSpreadBytes / ES, WARPS = kSpreadThreads / 32;
    constexpr int U = DOT ? 8 : kMaxTopk;              // entries at a time
    __shared__ __align__(128) char buf[DOT ? 1 + U : 1][kSpreadPitch];
    __shared__ Entries e;
    __shared__ float part[WARPS][kMaxTopk];
    __shared__ __align__(8) uint64_t bar_store;
    __shared__ int s_n;
    const uint32_t bar = smem_u32(&bar_store);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    griddep_launch_dependents();
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbarrier_init_cluster();
    }
    griddep_wait();
    if (warp == 0) {
        const int n = live_entries(e, pos, weights, ldw, t, k, rows, lane);
        if (lane == 0) s_n = n;
    }
    if constexpr (DOT)
        for (int i = tid; i < WARPS * kMaxTopk; i += kSpreadThreads) part[0][i] = 0.f;
    __syncthreads();
    const int n = s_n, chunks = (H + PER - 1) / PER;
    const uintptr_t glo = reinterpret_cast<uintptr_t>(G), ghi = glo + (uintptr_t)((T - 1) * ldg_bytes + (int64_t)H * ES);
    const uintptr_t ylo = reinterpret_cast<uintptr_t>(Ys), yhi = ylo + (uintptr_t)((rows - 1) * ldys_bytes + (int64_t)H * ES);
    int phase = 0;
    for (int j0 = 0; j0 < n; j0 += U) {
        const int m = min(U, n - j0);
        const int share = m >= WARPS ? 1 : m >= 2 ? 2 : WARPS, at_once = WARPS / share;    // warps per row, rows at once
        float dot[2] = {0.f, 0.f};
        for (int c = blockIdx.y; c < chunks; c += gridDim.y) {
            const int first = c * PER, len = min(H - first, PER);
            const int sources = DOT ? 1 + m : 1;
            // row s of the sources, from `first` on
            auto source = [&](int s) {
                return s == 0 ? glo + (uintptr_t)(t * ldg_bytes + (int64_t)first * ES)
                              : ylo + (uintptr_t)((int64_t)e.p[j0 + s - 1] * ldys_bytes + (int64_t)first * ES);
            };
            bool inside = true;        // whole pieces lie inside G and Ys; the same for every thread
            uint32_t bytes = 0;
            for (int s = 0; s < sources; ++s) {
                const uintptr_t a = source(s), a0 = a & ~(uintptr_t)15, a1 = (a + (uintptr_t)(len * ES) + 15) & ~(uintptr_t)15;
                inside = inside && a0 >= (s ? ylo : glo) && a1 <= (s ? yhi : ghi);
                bytes += (uint32_t)(a1 - a0);
            }
            if (inside) {
                if (tid == 0) {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(bar, bytes);
                    for (int s = 0; s < sources; ++s) {
                        const uintptr_t a = source(s), a0 = a & ~(uintptr_t)15, a1 = (a + (uintptr_t)(len * ES) + 15) & ~(uintptr_t)15;
                        bulk_copy_g2s(smem_u32(buf[s] + 16), reinterpret_cast<const void *>(a0), (uint32_t)(a1 - a0), bar);
                    }
                }
                const bool got = mbar_wait_bounded(bar, (uint32_t)(phase & 1), budget_ns);
                if (__syncthreads_or(got ? 0 : 1)) {
                    if (tid == 0) {
                        report_status(status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitX);
                        // the copies land before the CTA leaves
                        if (!mbar_wait_bounded(bar, (uint32_t)(phase & 1), kBulkDrainNs))
                            report_status(status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
                    }
                    __syncthreads();
                    return;
                }
                ++phase;
            } else {
                for (int s = 0; s < sources; ++s) {
                    const uintptr_t a = source(s);
                    char *to = buf[s] + 16 + (a & 15);
                    for (int i = tid; i < len; i += kSpreadThreads) {
                        if constexpr (B16) *reinterpret_cast<uint16_t *>(to + 2 * i) = ldg_u16(reinterpret_cast<const char *>(a) + 2 * i);
                        else *reinterpret_cast<float *>(to + 4 * i) = __ldcg(reinterpret_cast<const float *>(a) + i);
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int h = 0; h < (DOT ? U / WARPS : 1); ++h) {
                for (int q = at_once * h + warp / share; q < m; q += DOT ? U : at_once) {
                    const float w = e.w[j0 + q];
                    char *d = out + (int64_t)e.p[j0 + q] * ldo_bytes + (int64_t)first * ES;
                    const int off = (int)(reinterpret_cast<uintptr_t>(d) & 15);
                    const int pieces = (off + len * ES + 15) / 16;
                    const char *g = buf[0] + 16 + (source(0) & 15) - off;
                    const char *y = DOT ? buf[1 + (DOT ? q : 0)] + 16 + (source(1 + q) & 15) - off : g;
                    const int gs = (int)(smem_u32(g) & 15), ys = (int)(smem_u32(y) & 15);
                    d -= off;
                    g -= gs;
                    y -= ys;
#pragma unroll 2
                    for (int i = lane + 32 * (warp % share); i < pieces; i += 32 * share) {
                        const uint4 gv = shifted16(*reinterpret_cast<const uint4 *>(g + 16 * i),
                                                   *reinterpret_cast<const uint4 *>(g + 16 * i + 16), gs);
                        const int el = (16 * i - off) / ES;            // of the chunk; exact: off is whole elements
                        const bool whole = el >= 0 && el + NE <= len;
                        Raw<16> r, o;
                        r.w[0] = gv.x; r.w[1] = gv.y; r.w[2] = gv.z; r.w[3] = gv.w;
                        o = r;
                        if constexpr (MODE != kCopy) {
                            float v[NE];
#pragma unroll
                            for (int x = 0; x < NE; ++x) v[x] = w * raw_el<B16, 16>(r, x);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                if constexpr (B16) o.w[x] = pack_bf16(v[2 * x], v[2 * x + 1]);
                                else o.w[x] = __float_as_uint(v[x]);
                            }
                        }
                        if constexpr (DOT) {
                            const uint4 yv = shifted16(*reinterpret_cast<const uint4 *>(y + 16 * i),
                                                       *reinterpret_cast<const uint4 *>(y + 16 * i + 16), ys);
                            Raw<16> z;
                            z.w[0] = yv.x; z.w[1] = yv.y; z.w[2] = yv.z; z.w[3] = yv.w;
#pragma unroll
                            for (int x = 0; x < NE; ++x)
                                if (whole || (unsigned)(el + x) < (unsigned)len)
                                    dot[h] = fmaf(raw_el<B16, 16>(r, x), raw_el<B16, 16>(z, x), dot[h]);
                        }
                        if (whole) {
                            *reinterpret_cast<uint4 *>(d + 16 * i) = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
                        } else {
#pragma unroll
                            for (int x = 0; x < NE; ++x)
                                if ((unsigned)(el + x) < (unsigned)len) {
                                    if constexpr (B16) *reinterpret_cast<uint16_t *>(d + 16 * i + 2 * x) = (uint16_t)(o.w[x >> 1] >> (16 * (x & 1)));
                                    else *reinterpret_cast<uint32_t *>(d + 16 * i + 4 * x) = o.w[x];
                                }
                        }
                    }
                }
            }
            __syncthreads();           // the chunk is read before the next one lands
        }
        if constexpr (DOT) {
#pragma unroll
            for (int h = 0; h < U / WARPS; ++h) {
                const int q = at_once * h + warp / share;
                const float s = warp_sum(dot[h]);
                if (q < m && lane == 0) part[warp % share][e.j[j0 + q]] = s;
            }
        }
    }
    if constexpr (DOT) {
        __syncthreads();
        if (tid < k) {
            float s = part[0][tid];
            for (int i = 1; i < WARPS; ++i) s += part[i][tid];
            dw[t * lddw + tid] = s;
        }
    }
}

// ------------------------------------------------------------------ launches
uintptr_t u(const void *p) { return reinterpret_cast<uintptr_t>(p); }

cudaError_t launch(const void *fn, dim3 grid, int threads, int smem, cudaStream_t stream, bool pdl, int cluster,
                   void **args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Widest vector that every row start and the row length allow.
int vec_bytes(int64_t row_bytes, int el_bytes, uintptr_t all) {
    for (int v = 16; v > el_bytes; v >>= 1)
        if (all % v == 0 && row_bytes % v == 0) return v;
    return el_bytes;
}

// CTAs along a row of `nvec` vectors for T tokens: two CTAs per SM while each
// still has a vector per thread.
int row_chunks(int64_t T, int nvec, int num_sms) {
    const int64_t want = (2ll * num_sms + T - 1) / T;
    const int64_t most = (nvec + kRowThreads - 1) / kRowThreads;
    return (int)(want < most ? want : (most > 0 ? most : 1));
}

// Whether the one-launch form is taken: its work grows with the square of the
// entries, divided by the entries a CTA counts for.  GB300, one launch against
// sort and copy, us: 192 x 8 entries 5.5 and 8.8, 256 x 8 7.9 and 9.3, 384 x 8
// 10.8 and 8.8, 2000 x 1 12.5 and 9.5.
bool few_entries(int n, int k) { return n <= 1024 || (n <= 2048 && k >= 4); }

template <bool B16, Spread MODE>
cudaError_t spread_bulk(const CombineGradArgs &a, const CallCtx &c, cudaStream_t stream) {
    const int b = B16 ? 2 : 4;
    const char *G = static_cast<const char *>(a.dY), *Ys = static_cast<const char *>(a.Ys);
    char *out = static_cast<char *>(a.dYs);
    int64_t ldg = a.lddy * b, ldys = a.ldys * b, ldo = a.lddys * b, ldw = a.ldw, lddw = a.lddw;
    int rows = a.rows, T = a.T, k = a.k, H = a.H;
    const int32_t *pos = a.pos;
    const float *w = a.weights;
    float *dw = a.dweights;
    int *status = c.status;
    uint64_t budget = c.budget_ns;
    void *args[] = {&G, &ldg, &T, &Ys, &ldys, &rows, &pos, &w, &ldw, &k, &H, &out, &ldo, &dw, &lddw, &status, &budget};
    const int chunks = MODE == kScaleDot ? 1 : (H + kSpreadBytes / b - 1) / (kSpreadBytes / b);
    return launch((const void *)spread_bulk_kernel<B16, MODE>, dim3(T, chunks), kSpreadThreads, 0, stream, c.pdl, 1, args);
}

template <int VB>
cudaError_t dispatch_vec(const DispatchArgs &a, int nvec, const CallCtx &c, cudaStream_t stream) {
    const int num_sms = c.num_sms;
    const bool pdl = c.pdl;
    const char *X = static_cast<const char *>(a.X);
    char *Xs = static_cast<char *>(a.Xs);
    int64_t ldx = a.ldx * a.el_bytes, ldxs = a.ldxs * a.el_bytes, ldid = a.ldid;
    int T = a.T, k = a.k, E = a.E, n = a.T * a.k;
    const int32_t *ids = a.ids;
    int32_t *pos = a.pos, *order = a.order, *offsets = a.offsets;
    if (few_entries(n, k)) {
        const int smem = 4 * (n > E ? n : E);
        void *args[] = {&ids, &ldid, &X, &ldx, &T, &k, &E, &nvec, &pos, &order, &offsets, &Xs, &ldxs};
        return launch((const void *)dispatch_small_kernel<VB>, dim3(T + 1, T ? row_chunks(T, nvec, num_sms) : 1),
                      kRowThreads, smem, stream, pdl, 1, args);
    }
    int W = kSortSmem / 4 / E - 2;
    if (W > 32) W = 32;
    void *args[] = {&ids, &ldid, &k, &n, &E, &pos, &order, &offsets};
    cudaError_t e = launch((const void *)expert_sort_kernel, dim3(kSortCluster), 32 * W, 4 * (W + 2) * E, stream, pdl,
                           kSortCluster, args);
    if (e != cudaSuccess || nvec == 0) return e;
    if constexpr (VB < 8) {
        // a chunk brought to shared memory pays where it is stored more than a few times.  GB300, us by elements
        // and this way: 3001 x 6 x 2881 bf16 40 and 33, fp32 63 and 50; 2500 x 3 x 2001 bf16 15.0 and 17.7
        if (k >= 4) {
            const CombineGradArgs g{X, a.ldx, nullptr, 0, n, pos, nullptr, 0, T, k, a.H, a.el_bytes == 2, Xs, a.ldxs, nullptr, 0};
            return g.b16 ? spread_bulk<true, kCopy>(g, c, stream) : spread_bulk<false, kCopy>(g, c, stream);
        }
    }
    const int32_t *cpos = pos;
    void *cargs[] = {&cpos, &X, &ldx, &k, &nvec, &Xs, &ldxs};
    return launch((const void *)dispatch_copy_kernel<VB>, dim3(T, row_chunks(T, nvec, num_sms)), kRowThreads, 0,
                  stream, pdl, 1, cargs);
}

// Pieces of a row of `steps` steps of a warp: eight rounds of warps, so that the
// last one's end is short, two steps in each; single steps only where even
// these leave SMs without warps.
int row_pieces(int T, int steps, int num_sms) {
    const int64_t few = (20ll * num_sms + T - 1) / T, many = (160ll * num_sms + T - 1) / T;
    int S = (int)(many < (steps + 1) / 2 ? many : (steps + 1) / 2);
    if (S < few) S = (int)(few < steps ? few : steps);
    return S < 1 ? 1 : S;
}

template <bool IN16, bool OUT16, int VB>
cudaError_t combine_vec(const CombineArgs &a, int num_sms, cudaStream_t stream, bool pdl) {
    const char *Ys = static_cast<const char *>(a.Ys);
    char *Y = static_cast<char *>(a.Y);
    int64_t ldys = a.ldys * (IN16 ? 2 : 4), ldy = a.ldy * (OUT16 ? 2 : 4), ldw = a.ldw;
    int rows = a.rows, T = a.T, k = a.k, nvec = (int)((int64_t)a.H * (IN16 ? 2 : 4) / VB);
    const int32_t *pos = a.pos;
    const float *w = a.weights;
    constexpr int step = 32 * (VB >= 8 ? 2 : 4);
    int S = row_pieces(T, (nvec + step - 1) / step, num_sms);
    const int64_t jobs = (int64_t)T * S;
    void *args[] = {&Ys, &ldys, &rows, &pos, &w, &ldw, &T, &k, &nvec, &S, &Y, &ldy};
    return launch((const void *)combine_kernel<IN16, OUT16, VB>, dim3((unsigned)((jobs + 3) / 4)), 128, 0, stream, pdl, 1,
                  args);
}
template <bool IN16, bool OUT16>
cudaError_t combine_bulk(const CombineArgs &a, const CallCtx &c, cudaStream_t stream) {
    const char *Ys = static_cast<const char *>(a.Ys);
    char *Y = static_cast<char *>(a.Y);
    int64_t ldys = a.ldys * (IN16 ? 2 : 4), ldy = a.ldy * (OUT16 ? 2 : 4), ldw = a.ldw;
    int rows = a.rows, k = a.k, H = a.H;
    const int32_t *pos = a.pos;
    const float *w = a.weights;
    int *status = c.status;
    uint64_t budget = c.budget_ns;
    constexpr int per = kBulkBytes / (IN16 ? 2 : 4);
    // the grid's y holds 65535 tokens
    for (int t0 = 0; t0 < a.T; t0 += 65535) {
        const int n = a.T - t0 < 65535 ? a.T - t0 : 65535;
        void *args[] = {&Ys, &ldys, &rows, &pos, &w, &ldw, &k, &H, &Y, &ldy, &status, &budget};
        const cudaError_t e = launch((const void *)combine_bulk_kernel<IN16, OUT16>, dim3((H + per - 1) / per, n),
                                     kBulkThreads, 0, stream, c.pdl, 1, args);
        if (e != cudaSuccess) return e;
        if (pos) pos += (int64_t)n * k;
        if (w) w += (int64_t)n * ldw;
        Y += (int64_t)n * ldy;
    }
    return cudaSuccess;
}
template <bool IN16, bool OUT16>
cudaError_t combine_types(const CombineArgs &a, const CallCtx &c, cudaStream_t stream) {
    const int num_sms = c.num_sms;
    const bool pdl = c.pdl;
    constexpr int ib = IN16 ? 2 : 4, ob = OUT16 ? 2 : 4;
    // the widest load at which every row of Ys starts, ends and is stored aligned
    const uintptr_t in = u(a.Ys) | (uintptr_t)(a.ldys * ib), out = u(a.Y) | (uintptr_t)(a.ldy * ob);
    auto fits = [&](int vb) {
        const int st = vb / ib * ob;
        return in % vb == 0 && (int64_t)a.H * ib % vb == 0 && out % (st > 16 ? 16 : st) == 0;
    };
    if (fits(16)) return combine_vec<IN16, OUT16, 16>(a, num_sms, stream, pdl);
    if (fits(8)) return combine_vec<IN16, OUT16, 8>(a, num_sms, stream, pdl);
    if constexpr (IN16) {
        if (fits(4)) return combine_vec<IN16, OUT16, 4>(a, num_sms, stream, pdl);
    }
    return combine_bulk<IN16, OUT16>(a, c, stream);
}

template <bool B16, int VB, bool DW>
cudaError_t grad_as(const CombineGradArgs &a, int num_sms, cudaStream_t stream, bool pdl) {
    const int b = B16 ? 2 : 4;
    const char *dY = static_cast<const char *>(a.dY), *Ys = static_cast<const char *>(a.Ys);
    char *dYs = static_cast<char *>(a.dYs);
    int64_t lddy = a.lddy * b, ldys = a.ldys * b, lddys = a.lddys * b, ldw = a.ldw, lddw = a.lddw;
    int rows = a.rows, T = a.T, k = a.k, nvec = (int)((int64_t)a.H * b / VB);
    const int32_t *pos = a.pos;
    const float *w = a.weights;
    float *dw = a.dweights;
    // warps per token: as few as fill the SMs
    int S = 1;
    while (S < kRowThreads / 32 && (int64_t)T * S < 32ll * num_sms) S *= 2;
    void *args[] = {&dY, &lddy, &Ys, &ldys, &rows, &pos, &w, &ldw, &T, &k, &nvec, &S, &dYs, &lddys, &dw, &lddw};
    const int per = kRowThreads / 32 / S;
    return launch((const void *)combine_grad_kernel<B16, VB, DW>, dim3((T + per - 1) / per), kRowThreads, 0, stream, pdl,
                  1, args);
}
template <bool B16, bool DW>
cudaError_t grad_types(const CombineGradArgs &a, const CallCtx &c, cudaStream_t stream) {
    const int num_sms = c.num_sms;
    const bool pdl = c.pdl;
    constexpr int b = B16 ? 2 : 4;
    const uintptr_t all = u(a.dY) | u(a.dYs) | (uintptr_t)(a.lddy * b) | (uintptr_t)(a.lddys * b) |
                          (DW ? u(a.Ys) | (uintptr_t)(a.ldys * b) : 0);
    const int vb = vec_bytes((int64_t)a.H * b, b, all);
    // GB300, us by elements and this way: 3001 x 6 x 2881 bf16 250 and 70, fp32 88 and 80; one token x 8 x 501
    // bf16 5.0 and 8.6, 40 x 8 x 7001 29 and 23
    if (vb == b && a.T >= (B16 ? 32 : 2 * num_sms)) return spread_bulk<B16, DW ? kScaleDot : kScale>(a, c, stream);
    switch (vb) {
        case 16: return grad_as<B16, 16, DW>(a, num_sms, stream, pdl);
        case 8: return grad_as<B16, 8, DW>(a, num_sms, stream, pdl);
        case 4: return grad_as<B16, 4, DW>(a, num_sms, stream, pdl);
        default: return grad_as<B16, B16 ? 2 : 4, DW>(a, num_sms, stream, pdl);
    }
}

}  // namespace

cudaError_t expert_rows_prepare() { return set_max_dyn_smem(&expert_sort_kernel); }

cudaError_t launch_dispatch(const DispatchArgs &a, const CallCtx &c, cudaStream_t stream) {
    const int64_t row = (int64_t)a.H * a.el_bytes;
    const bool rows = a.X != nullptr && row > 0;
    const int vb = rows ? vec_bytes(row, a.el_bytes,
                                    u(a.X) | u(a.Xs) | (uintptr_t)(a.ldx * a.el_bytes) | (uintptr_t)(a.ldxs * a.el_bytes))
                        : 16;
    const int nvec = rows ? (int)(row / vb) : 0;
    switch (vb) {
        case 16: return dispatch_vec<16>(a, nvec, c, stream);
        case 8: return dispatch_vec<8>(a, nvec, c, stream);
        case 4: return dispatch_vec<4>(a, nvec, c, stream);
        default: return dispatch_vec<2>(a, nvec, c, stream);
    }
}

cudaError_t launch_combine(const CombineArgs &a, const CallCtx &c, cudaStream_t stream) {
    if (a.in16) return a.out16 ? combine_types<true, true>(a, c, stream) : combine_types<true, false>(a, c, stream);
    return a.out16 ? combine_types<false, true>(a, c, stream) : combine_types<false, false>(a, c, stream);
}

cudaError_t launch_combine_grad(const CombineGradArgs &a, const CallCtx &c, cudaStream_t stream) {
    if (a.b16) return a.dweights ? grad_types<true, true>(a, c, stream) : grad_types<true, false>(a, c, stream);
    return a.dweights ? grad_types<false, true>(a, c, stream) : grad_types<false, false>(a, c, stream);
}

}  // namespace skinny
