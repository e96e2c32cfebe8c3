// experts_tc.cu -- the experts' products on the fifth-generation tensor cores:
//     Y[r,n] = sum_k X[r,k] W[e][n][k]      offsets[e] <= r < offsets[e+1]
// or, with SwiGLU, g / (1 + exp(-g)) * u of the rows n and N + n of W[e].
//
// At decode an expert has a few rows, so the weights of the experts that occur
// are the traffic: the kernel is a stream of W through shared memory, once.
//   * Work split.  An expert's rows of W are 16-row groups (SwiGLU: a group is 8
//     gates and their 8 ups), dealt evenly to tiles of at most 8 groups; the
//     tiles of all experts that have rows are dealt evenly to the CTAs, two per
//     SM.  The tiles' size is chosen in the kernel, where the number of experts
//     that have rows is known.  (Equal pieces of the line of groups, whatever
//     the tiles, left CTAs whose piece met an expert's end with twice the
//     stages: 32 experts, 2 x 512 x 4096, 16 rows each: 80 us.)
//   * Per tile, W (up to 128 rows) is the MMA's M side, up to 64 rows of X its
//     N side (16, 32, 48 or 64, as the expert has rows).  An expert with more
//     than 64 rows is walked again for the next 64, its tile of W then in L2.
//   * Thread 0 loads 64-element boxes of W and X by tensor-map TMA into a ring,
//     a tile's height of W in one box (there is a map for each height: with
//     boxes of 128, 64, 32, 16 and 8 rows put together the copies' number, about
//     0.1 us each, was the limit of short tiles);
//     thread 32 issues tcgen05.mma into four sets of tensor-memory
//     accumulators in rotation, at most 16 MMAs a set; warps 2..5 add each set
//     into fp32 registers (one row of W per thread, its tokens in registers)
//     and store the tile at its end: the same bounded chains and rounded adds
//     as the shared projections (the tensor core's own sums are biased).
//   * SwiGLU: a tile is up to 64 gates on the MMA's first rows and their ups on
//     as many rows behind them; at its end the ups go through shared memory to
//     the gates' threads.
// Every wait is bounded.  A wait that gives up records an error and the CTA
// winds down, storing no tile from there on: copies in flight and issued MMAs are waited for
// (bounded) and the draining warps still meet at every barrier.
#include <cuda.h>
#include <type_traits>

#include "common.cuh"
#include "experts_gemm.h"
#include "tcgen05.cuh"
#include "tma_stack.cuh"

namespace skinny {
namespace {

constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
enum : int { kWaitAcc = 5, kWaitAccEmpty = 6 };
constexpr int kThreads = 192;          // TMA warp, MMA warp, four draining warps
constexpr int kGroups = 8;             // groups per tile: W boxes of 1 to 8 of them
constexpr int kXBoxes = 4;             // X boxes of 16, 32, 48, 64 rows
constexpr int kSets = 4;               // accumulator sets in rotation
constexpr int kSetCols = 64;           // fp32 columns of a set
constexpr int kTmemCols = kSets * kSetCols;
constexpr int kCtasPerSm = 2;          // 2 x 256 columns fill an SM's tensor memory

struct Maps {
    CUtensorMap w[kGroups];            // box heights of 1 to 8 groups (16 rows, SwiGLU 8)
    CUtensorMap x[kXBoxes];
};

struct Params {
    const int32_t *offsets;
    void *Y;
    int64_t ldy;
    int rows, E, N, K;
    int out_bf16;
    int *status;
    uint64_t budget_ns;
};

// A stage holds up to 128 rows of W and 64 rows of X, 64 elements of K each; a
// tile of half or a quarter of that takes 2 or 4 times the elements of K per
// stage, so that short tiles keep as many bytes in flight and a CTA whose piece
// meets an expert's end runs no more stages than the others (GB300, 16 experts,
// 2048 x 2048, 2 rows each: 43 us with one box a stage).
constexpr int kNT = 64;
constexpr int kStage = (128 + kNT) * 128;
constexpr int kStages = 4;
__host__ __device__ inline int tile_boxes(int groups, int xb) {
    return groups <= 2 && xb <= 1 ? 4 : groups <= 4 && xb <= 2 ? 2 : 1;
}
constexpr int kExBytes = 16 * 64 * 4;                  // SwiGLU: 16 tokens of 64 ups
constexpr int kBarBytes = 8 * (2 * kStages + 2 * kSets + 1);
// After the ring: barriers, tensor-memory address, flags, the exchange, the
// experts' rows and list; 12 KB at least, for an MMA reads 128 rows from each
// box of W, past the stage's end in the last one (those rows are not stored).
int smem_bytes(int E) {
    int tail = kBarBytes + 16 + kExBytes + 4 * (E + 1) + 2 * E + 16;
    if (tail < 12 * 1024) tail = 12 * 1024;
    return 1024 + kStages * kStage + tail;             // 110 KB: two CTAs on an SM, as tensor memory holds
}
// Tensor memory is allocated behind griddep_wait, when CTAs of the next kernel may be on the SM and hold theirs.  An
// SM always has columns for its CTAs, since those of every kernel that takes some (here and tmem_gemm.cu) take 256 and
// ask for so much shared memory that no three fit (with the 1 KB that each CTA is charged beside it).
static_assert(1024 + kStages * kStage + 12 * 1024 >= kTcMinSmem && 3 * (kTcMinSmem + 1024) > 228 * 1024,
              "at most two CTAs with tensor memory on an SM");

// Groups [g, g + ng) of expert e.
struct Tile {
    int e, g, ng, row0, count;
    // X boxes of 16 rows for the rows from m0 on
    __device__ __forceinline__ int xb(int m0) const { return (min(kNT, count - m0) + 15) / 16; }
};

// Walks a CTA's tiles [i, i1); every role walks them for itself.
struct Walk {
    int i, i1;
    int GN, nt;                        // groups and tiles per expert
    const int *row;                    // clamped offsets [E + 1]
    const uint16_t *active;            // the experts that have rows
    __device__ __forceinline__ bool next(Tile &t) {
        if (i >= i1) return false;
        const int a = i / nt, at = i - a * nt;
        t.g = (int)((int64_t)at * GN / nt);
        t.ng = (int)((int64_t)(at + 1) * GN / nt) - t.g;
        t.e = active[a];
        t.row0 = row[t.e];
        t.count = row[t.e + 1] - t.row0;
        ++i;
        return true;
    }
};

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
experts_tc_kernel(const __grid_constant__ Maps maps, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    griddep_launch_dependents();
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t bars = base + kStages * kStage;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto accf = [&](int b) { return bars + 8u * (2 * kStages + b); };
    auto acce = [&](int b) { return bars + 8u * (2 * kStages + kSets + b); };
    const uint32_t done = bars + 8u * (2 * kStages + 2 * kSets);
    uint8_t *tail = smem + kStages * kStage + kBarBytes;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int *mma_ok = reinterpret_cast<volatile int *>(tail + 4);
    float *ex = reinterpret_cast<float *>(tail + 16);
    int *row = reinterpret_cast<int *>(tail + 16 + kExBytes);
    uint16_t *active = reinterpret_cast<uint16_t *>(row + p.E + 1);
    __shared__ int s_warp[kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kGroups; ++i) prefetch_tensormap(&maps.w[i]);
        for (int i = 0; i < kXBoxes; ++i) prefetch_tensormap(&maps.x[i]);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < kSets; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 4);
        }
        mbar_init(done, 1);
        *mma_ok = 0;
        fence_mbarrier_init_cluster();
    }
    griddep_wait();                    // the offsets and rows come from the preceding kernel

    // the experts that have rows, in order
    const int E = p.E;
    for (int e = tid; e <= E; e += kThreads) row[e] = max(0, min(p.rows, __ldcg(p.offsets + e)));
    __syncthreads();
    int found = 0;
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = e0 + tid;
        const bool has = e < E && row[e + 1] > row[e];
        const unsigned ball = __ballot_sync(0xFFFFFFFFu, has);
        if (lane == 0) s_warp[warp] = __popc(ball);
        __syncthreads();
        int before = found;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            found += s_warp[w];
        }
        if (has) active[before + __popc(ball & ((1u << lane) - 1))] = (uint16_t)e;
        __syncthreads();
    }
    constexpr int kRows = SWIGLU ? 8 : 16;             // rows of W's first half per group
    const int GN = (p.N + kRows - 1) / kRows;
    // tiles per expert: the number for which the CTA with the most tiles has the
    // least to do, a tile costing its groups and about one and a half of fixed work
    int nt = 0;
    float least = 0.f;
    for (int ts = kGroups; ts >= 1; --ts) {
        const int n = (GN + ts - 1) / ts;
        const int64_t rounds = ((int64_t)found * n + gridDim.x - 1) / gridDim.x;
        const float cost = (float)rounds * ((float)((GN + n - 1) / n) + 1.5f);
        if (nt == 0 || cost < least) { nt = n; least = cost; }
    }
    const int64_t tiles = (int64_t)found * nt;
    Walk walk{(int)(tiles * blockIdx.x / gridDim.x), (int)(tiles * (blockIdx.x + 1) / gridDim.x), GN, nt, row, active};
    if (walk.i >= walk.i1) return;     // the whole CTA

    const int boxes = (p.K + 63) / 64;

    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer
            int64_t i = 0;             // stage number
            bool go = true;
            Tile t;
            while (go && walk.next(t)) {
                const int n0 = kRows * t.g;
                for (int m0 = 0; go && m0 < t.count; m0 += kNT) {
                    const int xb = t.xb(m0), kb = tile_boxes(t.ng, xb);
                    for (int k0 = 0; k0 < boxes; k0 += kb, ++i) {
                        const int s = (int)(i % kStages);
                        if (i >= kStages &&
                            !mbar_wait_bounded(empty(s), (uint32_t)((i / kStages - 1) & 1), p.budget_ns)) {
                            report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitProducerEmpty);
                            go = false;
                            break;
                        }
                        const int nb = min(kb, boxes - k0);
                        mbar_arrive_expect_tx(full(s), (uint32_t)(nb * 16 * (t.ng + xb) * 128));
                        const uint32_t st = base + s * kStage;
                        for (int b = 0; b < nb; ++b) {
                            const int k = (k0 + b) * 64;
                            const uint32_t dst = st + b * (128 / kb) * 128;
                            tma_load_stack(dst, &maps.w[t.ng - 1], k, n0, t.e, full(s));
                            if (SWIGLU) tma_load_stack(dst + (64 / kb) * 128, &maps.w[t.ng - 1], k, p.N + n0, t.e, full(s));
                            tma_load_2d(st + 128 * 128 + b * (kNT / kb) * 128, &maps.x[xb - 1], k, t.row0 + m0, full(s));
                        }
                    }
                }
            }
            // every copy issued has landed before the CTA exits
            for (int64_t j = i > kStages ? i - kStages : 0; j < i; ++j)
                if (!mbar_wait_bounded(full((int)(j % kStages)), (uint32_t)((j / kStages) & 1), kDrainNs))
                    report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
        }
        __syncwarp();
    } else if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
        tc_fence_before();
        named_bar_sync(1, kThreads - 32);
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        if (lane == 0) {
            // ---- MMA issuer
            int64_t i = 0, c = 0;      // stage and chunk number
            bool go = true;
            Tile t;
            while (go && walk.next(t)) {
                for (int m0 = 0; go && m0 < t.count; m0 += kNT) {
                    const int xb = t.xb(m0), kb = tile_boxes(t.ng, xb);
                    const uint32_t n = 16u * (uint32_t)xb;
                    const uint32_t P = kSetCols / n;   // accumulators of a set, taken in turn
                    const uint32_t idesc = idesc_bf16_n<128>(n);
                    for (int k0 = 0; k0 < boxes; k0 += kb, ++i) {
                        const int s = (int)(i % kStages), b = (int)(c % kSets);
                        if (k0 % 4 == 0 && c >= kSets &&
                            !mbar_wait_bounded(acce(b), (uint32_t)((c / kSets - 1) & 1), p.budget_ns)) {
                            report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAccEmpty);
                            go = false;
                            break;
                        }
                        if (!mbar_wait_bounded(full(s), (uint32_t)((i / kStages) & 1), p.budget_ns)) {
                            report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitConsumerFull);
                            go = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t st = base + s * kStage;
                        const int nb = min(kb, boxes - k0);
                        uint32_t q = (uint32_t)(k0 % 4) * 4;   // a set takes four boxes: 16 MMAs
                        for (int bx = 0; bx < nb; ++bx)
#pragma unroll
                            for (int j = 0; j < 4; ++j, ++q)
                                umma_bf16(tmem + b * kSetCols + (q % P) * n, sw128_desc(st + bx * (128 / kb) * 128 + 32 * j),
                                          sw128_desc(st + 128 * 128 + bx * (kNT / kb) * 128 + 32 * j), idesc,
                                          q < P ? 0u : 1u);
                        umma_commit(empty(s));
                        if ((k0 + nb) % 4 == 0 || k0 + nb == boxes) {
                            umma_commit(accf(b));
                            ++c;
                        }
                    }
                }
            }
            umma_commit(done);
            if (mbar_wait_bounded(done, 0, kDrainNs)) *mma_ok = 1;
            else report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
        }
        __syncwarp();
    } else {
        // ---- draining warps: lane quarter q of tensor memory
        named_bar_sync(1, kThreads - 32);
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        const int q = warp & 3;
        const int arow = 32 * q + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
        int64_t c = 0;
        bool ok = true;
        auto tile = [&](auto XBc, const Tile &t, int m0) {
            constexpr int XB = decltype(XBc)::value;
            constexpr int P = kSetCols / (16 * XB);
            float acc[16 * XB];
#pragma unroll
            for (int j = 0; j < 16 * XB; ++j) acc[j] = 0.f;
            const int chunks = (boxes + 3) / 4;
            for (int k = 0; k < chunks; ++k, ++c) {
                const int b = (int)(c % kSets);
                if (ok) {
                    bool got = true;
                    if (lane == 0) got = mbar_wait_bounded(accf(b), (uint32_t)((c / kSets) & 1), p.budget_ns);
                    got = __shfl_sync(0xFFFFFFFFu, got ? 1 : 0, 0) != 0;
                    if (!got) {
                        if (lane == 0) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAcc);
                        ok = false;
                    }
                }
                if (!ok) continue;     // the barriers below are still met
                tc_fence_after();
                // the set's sums, in order (a chunk has four MMAs at least, P is four at most)
#pragma unroll
                for (int pp = 0; pp < P; ++pp) {
#pragma unroll
                    for (int cc = 0; cc < XB; ++cc) {
                        uint32_t r[16];
                        tmem_ld16_nowait(lane_base + (uint32_t)(b * kSetCols + pp * 16 * XB + 16 * cc), r);
                        tmem_ld_wait(r);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[16 * cc + j] += __uint_as_float(r[j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce(b));
            }
            const int cols = min(kNT, t.count - m0);
            const int64_t y0 = (int64_t)(t.row0 + m0) * p.ldy;
            if constexpr (!SWIGLU) {
                const int n = kRows * t.g + arow;
                if (ok && arow < kRows * t.ng && n < p.N) {
#pragma unroll
                    for (int m = 0; m < 16 * XB; ++m)
                        if (m < cols) store_y(p.Y, p.out_bf16, y0 + m * p.ldy + n, acc[m]);
                }
            } else {
                const int half = 64 / tile_boxes(t.ng, XB);          // the gates' rows, then the ups'
                const int n = kRows * t.g + arow;
                const bool live = arow < kRows * t.ng && n < p.N;
#pragma unroll
                for (int cc = 0; cc < XB; ++cc) {
                    if (arow >= half && arow < 2 * half) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) ex[j * 64 + arow - half] = acc[16 * cc + j];
                    }
                    __syncwarp();
                    named_bar_sync(2, 128);
                    if (live && ok) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float g = acc[16 * cc + j];
                            if (16 * cc + j < cols)
                                store_y(p.Y, p.out_bf16, y0 + (16 * cc + j) * p.ldy + n, g / (1.f + expf(-g)) * ex[j * 64 + arow]);
                        }
                    }
                    __syncwarp();
                    named_bar_sync(2, 128);
                }
            }
        };
        Tile t;
        while (walk.next(t)) {
            for (int m0 = 0; m0 < t.count; m0 += kNT) {
                switch (t.xb(m0)) {
                    case 1: tile(std::integral_constant<int, 1>{}, t, m0); break;
                    case 2: tile(std::integral_constant<int, 2>{}, t, m0); break;
                    case 3: tile(std::integral_constant<int, 3>{}, t, m0); break;
                    default: tile(std::integral_constant<int, 4>{}, t, m0); break;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (*mma_ok) tmem_dealloc(*tmem_slot, kTmemCols);
        // else an issued MMA may still write it: it stays allocated until the CTA exits
    }
}

using Kernel = void (*)(const Maps, const Params);
const Kernel kKernels[2] = {&experts_tc_kernel<false>, &experts_tc_kernel<true>};

}  // namespace

bool experts_tc_supported(const ExpertsArgs &a) {
    return a.K >= 1 && (reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.W)) % 16 == 0 &&
           a.ldx % 8 == 0 && a.ldw % 8 == 0 && a.ldwe % 8 == 0 && a.ldwe < (1ll << 38);
}

// The mma.sync kernel reads W at the rate of device memory while an expert has
// up to 8 rows and reads it again (from L2) for the next 8; this one holds 64
// rows but needs long lines to fill its tiles.  Measured on GB300, tcgen05
// against mma.sync (us): 256 experts 2048 x 2048, 1 row each on average 166 and
// 154, 2 rows 218 and 213; 7168 x 2048, 2 rows, unevenly 423 and 503; 32 experts
// 2048 x 2048, 16 rows 54 and 83; 8 experts 16 rows, 4096 x 1024 (2048 groups)
// 21 and 24, 2048 x 2048 (1024 groups) 27 and 24; 1 matrix 24576 x 1536, 64 rows
// (1536 groups) 28 and 50.  A tile's fill and its epilogue cost as much as about
// 256 elements of K: 19 experts, SwiGLU, 1242 x 64, 19 rows each 21.6 and 6.8, 18
// experts 3392 x 128, 7 rows 12.9 and 7.7, 10 experts 4000 x 192, 5 rows 12.1 and
// 6.7, 29 experts 6568 x 256, 5 rows 25.7 and 33.3.
bool experts_tc_faster(const ExpertsArgs &a, int num_sms) {
    const int per = a.swiglu ? 8 : 16;
    const int64_t groups = (int64_t)(a.rows < a.E ? a.rows : a.E) * ((a.N + per - 1) / per), ctas = (int64_t)kCtasPerSm * num_sms;
    if (a.K <= 192) return false;
    return (a.rows >= 2 * a.E && groups >= kGroups * ctas) || (a.rows >= 8 * a.E && groups >= 5 * ctas);
}

cudaError_t experts_tc_prepare() {
    for (int i = 0; i < 2; ++i) {
        const cudaError_t e = set_max_dyn_smem(kKernels[i]);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_experts_tc(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream) {
    Maps maps;
    const int64_t wrows = a.swiglu ? 2ll * a.N : a.N;
    const int kRows = a.swiglu ? 8 : 16;
    for (int h = 0; h < kGroups; ++h)
        if (!encode_bf16_stack(&maps.w[h], a.W, a.K, wrows, a.E, a.ldw, a.ldwe, kRows * (h + 1))) return cudaErrorInvalidValue;
    for (int h = 0; h < kXBoxes; ++h)
        if (!encode_bf16_2d(&maps.x[h], a.X, a.K, a.rows, a.ldx, 16 * (h + 1))) return cudaErrorInvalidValue;
    const Params p{a.offsets, a.Y, a.ldy, a.rows, a.E, a.N, a.K, a.out_bf16, c.status, c.budget_ns};
    const int64_t groups = (int64_t)(a.rows < a.E ? a.rows : a.E) * ((a.N + kRows - 1) / kRows);
    const int64_t most = (int64_t)kCtasPerSm * c.num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups < most ? groups : most), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(a.E);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kKernels[a.swiglu ? 1 : 0], maps, p);
}

}  // namespace skinny
