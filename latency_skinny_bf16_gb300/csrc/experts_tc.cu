// experts_tc.cu -- the experts' products on the fifth-generation tensor cores:
//     Y[r,n] = sum_k X[r,k] W[e][n][k]      offsets[e] <= r < offsets[e+1]
// or, with SwiGLU, g / (1 + exp(-g)) * u of the rows n and N + n of W[e].
//
// At decode an expert has a few rows, so the weights of the experts that occur
// are the traffic: the kernel is a stream of W through shared memory, once.
//   * Work split.  The rows of W of all experts that have rows form one line
//     of 8-row groups (an expert after the other; SwiGLU: a group is 8 gates
//     and their 8 ups).  The CTAs, two per SM, each take an equal piece of
//     that line, whatever the experts' number and sizes, and walk it in tiles
//     of at most 128 rows of W that do not cross an expert.
//   * Per tile, W (up to 128 rows) is the MMA's M side, up to NT rows of X its
//     N side (16, 32, 48 or 64, as the expert has rows).  An expert with more
//     than NT rows is walked again for the next NT, its tile of W then in L2.
//   * Thread 0 loads 64-element boxes of W and X by tensor-map TMA into a ring;
//     thread 32 issues tcgen05.mma into four sets of tensor-memory
//     accumulators in rotation, at most 16 MMAs a set; warps 2..5 add each set
//     into fp32 registers (one row of W per thread, its tokens in registers)
//     and store the tile at its end: the same bounded chains and rounded adds
//     as the shared projections (the tensor core's own sums are biased).
//   * SwiGLU: a tile is 64 gates on the MMA's rows 0..63 and their ups on rows
//     64..127; at its end the ups go through shared memory to the gates'
//     threads.
// Every wait is bounded.  A wait that gives up records an error and the CTA
// winds down without storing: copies in flight and issued MMAs are waited for
// (bounded) and the draining warps still meet at every barrier.
#include <cuda.h>
#include <type_traits>

#include "common.cuh"
#include "experts_gemm.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace skinny {
namespace {

constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
enum : int { kWaitAcc = 5, kWaitAccEmpty = 6 };
constexpr int kThreads = 192;          // TMA warp, MMA warp, four draining warps
constexpr int kHeights = 5;            // W boxes of 128, 64, 32, 16, 8 rows
constexpr int kSets = 4;               // accumulator sets in rotation
constexpr int kSetCols = 64;           // fp32 columns of a set
constexpr int kTmemCols = kSets * kSetCols;
constexpr int kCtasPerSm = 2;          // 2 x 256 columns fill an SM's tensor memory

struct Maps {
    CUtensorMap w[kHeights];
    CUtensorMap x;                     // boxes of 16 rows
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

// A stage: KB boxes of 128 rows of W, then KB boxes of NT rows of X.
template <int NT> struct Shape {
    static constexpr int kKB = 1;
    static constexpr int kStage = kKB * (128 + NT) * 128;
    static constexpr int kStages = (100 * 1024) / kStage;
    static constexpr int kChunk = 4 / kKB;             // stages per accumulator set: 16 MMAs
};
constexpr int kExBytes = 16 * 64 * 4;                  // SwiGLU: 16 tokens of 64 ups
// after the ring: barriers, tensor-memory address, flags, the exchange, the experts' rows and list
template <int NT> constexpr int bar_bytes() { return 8 * (2 * Shape<NT>::kStages + 2 * kSets + 1); }
template <int NT> int smem_bytes(int E) {
    const int b = 1024 + Shape<NT>::kStages * Shape<NT>::kStage + bar_bytes<NT>() + 16 + kExBytes + 4 * (E + 1) + 2 * E + 16;
    return b < 78 * 1024 ? 78 * 1024 : b;              // never three CTAs on an SM: tensor memory holds two
}

// A piece of the line of groups: groups [g, g + ng) of expert e.
struct Tile {
    int e, g, ng, row0, count;
};

// Walks a CTA's piece [i, i1) of the line; every role walks it for itself.
struct Walk {
    int64_t i, i1;
    int GN, most;                      // groups per expert, groups per tile
    const int *row;                    // clamped offsets [E + 1]
    const uint16_t *active;            // the experts that have rows
    __device__ __forceinline__ bool next(Tile &t) {
        if (i >= i1) return false;
        const int a = (int)(i / GN);
        t.g = (int)(i - (int64_t)a * GN);
        const int64_t end = (int64_t)(a + 1) * GN;
        const int left = (int)((i1 < end ? i1 : end) - i);
        const int n = (left + most - 1) / most;        // tiles left of this run, evenly
        t.ng = (left + n - 1) / n;
        t.e = active[a];
        t.row0 = row[t.e];
        t.count = row[t.e + 1] - t.row0;
        i += t.ng;
        return true;
    }
};

template <int NT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
experts_tc_kernel(const __grid_constant__ Maps maps, const Params p)
{
    using S = Shape<NT>;
    extern __shared__ uint8_t smem_raw[];
    griddep_launch_dependents();
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t bars = base + S::kStages * S::kStage;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S::kStages + s); };
    auto accf = [&](int b) { return bars + 8u * (2 * S::kStages + b); };
    auto acce = [&](int b) { return bars + 8u * (2 * S::kStages + kSets + b); };
    const uint32_t done = bars + 8u * (2 * S::kStages + 2 * kSets);
    uint8_t *tail = smem + S::kStages * S::kStage + bar_bytes<NT>();
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int *mma_ok = reinterpret_cast<volatile int *>(tail + 4);
    float *ex = reinterpret_cast<float *>(tail + 16);
    int *row = reinterpret_cast<int *>(tail + 16 + kExBytes);
    uint16_t *active = reinterpret_cast<uint16_t *>(row + p.E + 1);
    __shared__ int s_warp[kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kHeights; ++i) prefetch_tensormap(&maps.w[i]);
        prefetch_tensormap(&maps.x);
        for (int s = 0; s < S::kStages; ++s) {
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
    const int GN = (p.N + 7) / 8;
    const int64_t line = (int64_t)found * GN;
    Walk walk{line * blockIdx.x / gridDim.x, line * (blockIdx.x + 1) / gridDim.x, GN, SWIGLU ? 8 : 16, row, active};
    if (walk.i >= walk.i1) return;     // the whole CTA

    const int boxes = (p.K + 63) / 64;
    const int nk = (boxes + S::kKB - 1) / S::kKB;      // stages per tile and pass

    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer
            int64_t i = 0;             // stage number
            bool go = true;
            Tile t;
            while (go && walk.next(t)) {
                const int h = 8 * t.ng, n0 = 8 * t.g;
                for (int m0 = 0; go && m0 < t.count; m0 += NT) {
                    const int xb = (min(NT, t.count - m0) + 15) / 16;
                    for (int ks = 0; ks < nk; ++ks, ++i) {
                        const int s = (int)(i % S::kStages);
                        if (i >= S::kStages &&
                            !mbar_wait_bounded(empty(s), (uint32_t)((i / S::kStages - 1) & 1), p.budget_ns)) {
                            report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitProducerEmpty);
                            go = false;
                            break;
                        }
                        const int nb = min(S::kKB, boxes - ks * S::kKB);
                        mbar_arrive_expect_tx(full(s), (uint32_t)(nb * ((SWIGLU ? 2 : 1) * h + 16 * xb) * 128));
                        const uint32_t st = base + s * S::kStage;
                        for (int b = 0; b < nb; ++b) {
                            const int k = (ks * S::kKB + b) * 64;
                            int off = 0;
#pragma unroll
                            for (int q = 0; q < kHeights; ++q) {
                                const int height = 128 >> q;
                                if (SWIGLU && height == 128) continue;
                                if (h - off >= height) {
                                    const uint32_t dst = st + b * 128 * 128 + off * 128;
                                    tma_load_stack(dst, &maps.w[q], k, n0 + off, t.e, full(s));
                                    if (SWIGLU) tma_load_stack(dst + 64 * 128, &maps.w[q], k, p.N + n0 + off, t.e, full(s));
                                    off += height;
                                }
                            }
                            const uint32_t xd = st + S::kKB * 128 * 128 + b * NT * 128;
                            for (int x = 0; x < xb; ++x)
                                tma_load_2d(xd + x * 16 * 128, &maps.x, k, t.row0 + m0 + 16 * x, full(s));
                        }
                    }
                }
            }
            // every copy issued has landed before the CTA exits
            for (int64_t j = i > S::kStages ? i - S::kStages : 0; j < i; ++j)
                if (!mbar_wait_bounded(full((int)(j % S::kStages)), (uint32_t)((j / S::kStages) & 1), kDrainNs))
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
                for (int m0 = 0; go && m0 < t.count; m0 += NT) {
                    const uint32_t n = 16u * (uint32_t)((min(NT, t.count - m0) + 15) / 16);
                    const uint32_t P = kSetCols / n;   // accumulators of a set, taken in turn
                    const uint32_t idesc = idesc_bf16_n<128>(n);
                    for (int ks = 0; ks < nk; ++ks, ++i) {
                        const int s = (int)(i % S::kStages), b = (int)(c % kSets);
                        if (ks % S::kChunk == 0 && c >= kSets &&
                            !mbar_wait_bounded(acce(b), (uint32_t)((c / kSets - 1) & 1), p.budget_ns)) {
                            report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAccEmpty);
                            go = false;
                            break;
                        }
                        if (!mbar_wait_bounded(full(s), (uint32_t)((i / S::kStages) & 1), p.budget_ns)) {
                            report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitConsumerFull);
                            go = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t st = base + s * S::kStage;
                        const int nb = min(S::kKB, boxes - ks * S::kKB);
                        uint32_t q = (uint32_t)(ks % S::kChunk) * 4 * S::kKB;
                        for (int bx = 0; bx < nb; ++bx)
#pragma unroll
                            for (int j = 0; j < 4; ++j, ++q)
                                umma_bf16(tmem + b * kSetCols + (q % P) * n, sw128_desc(st + bx * 128 * 128 + 32 * j),
                                          sw128_desc(st + S::kKB * 128 * 128 + bx * NT * 128 + 32 * j), idesc,
                                          q < P ? 0u : 1u);
                        umma_commit(empty(s));
                        if (ks % S::kChunk == S::kChunk - 1 || ks == nk - 1) {
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
            const int chunks = (nk + S::kChunk - 1) / S::kChunk;
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
                // the chunk's MMAs reached min(P, MMAs) accumulators
                const int mmas = 4 * min(boxes - k * 4, 4);
#pragma unroll
                for (int pp = 0; pp < P; ++pp) {
                    if (pp >= mmas) break;
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
            const int cols = min(NT, t.count - m0);
            const int64_t y0 = (int64_t)(t.row0 + m0) * p.ldy;
            if constexpr (!SWIGLU) {
                const int n = 8 * t.g + arow;
                if (ok && arow < 8 * t.ng && n < p.N) {
#pragma unroll
                    for (int m = 0; m < 16 * XB; ++m)
                        if (m < cols) store_y(p.Y, p.out_bf16, y0 + m * p.ldy + n, acc[m]);
                }
            } else {
                const int n = 8 * t.g + (arow & 63);
                const bool live = (arow & 63) < 8 * t.ng && n < p.N;
#pragma unroll
                for (int cc = 0; cc < XB; ++cc) {
                    if (arow >= 64) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) ex[j * 64 + arow - 64] = acc[16 * cc + j];
                    }
                    __syncwarp();
                    named_bar_sync(2, 128);
                    if (arow < 64 && live && ok) {
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
            for (int m0 = 0; m0 < t.count; m0 += NT) {
                if constexpr (NT == 16) {
                    tile(std::integral_constant<int, 1>{}, t, m0);
                } else {
                    switch ((min(NT, t.count - m0) + 15) / 16) {
                        case 1: tile(std::integral_constant<int, 1>{}, t, m0); break;
                        case 2: tile(std::integral_constant<int, 2>{}, t, m0); break;
                        case 3: tile(std::integral_constant<int, 3>{}, t, m0); break;
                        default: tile(std::integral_constant<int, 4>{}, t, m0); break;
                    }
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
const Kernel kKernels[2][2] = {{&experts_tc_kernel<16, false>, &experts_tc_kernel<16, true>},
                               {&experts_tc_kernel<64, false>, &experts_tc_kernel<64, true>}};

}  // namespace

bool experts_tc_supported(const ExpertsArgs &a) {
    return a.K >= 1 && (reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.W)) % 16 == 0 &&
           a.ldx % 8 == 0 && a.ldw % 8 == 0 && a.ldwe % 8 == 0 && a.ldwe < (1ll << 38);
}

cudaError_t experts_tc_prepare() {
    for (int i = 0; i < 4; ++i) {
        const cudaError_t e = set_max_dyn_smem(kKernels[i >> 1][i & 1]);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_experts_tc(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream) {
    Maps maps;
    const int64_t wrows = a.swiglu ? 2ll * a.N : a.N;
    for (int h = 0; h < kHeights; ++h)
        if (!encode_bf16_stack(&maps.w[h], a.W, a.K, wrows, a.E, a.ldw, a.ldwe, 128 >> h)) return cudaErrorInvalidValue;
    if (!encode_bf16_2d(&maps.x, a.X, a.K, a.rows, a.ldx, 16)) return cudaErrorInvalidValue;
    const Params p{a.offsets, a.Y, a.ldy, a.rows, a.E, a.N, a.K, a.out_bf16, c.status, c.budget_ns};
    // up to 16 rows in all, no expert has more: the shape with the smaller share of X
    const int big = a.rows > 16;
    const int64_t groups = (int64_t)(a.rows < a.E ? a.rows : a.E) * ((a.N + 7) / 8);
    const int64_t most = (int64_t)kCtasPerSm * c.num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups < most ? groups : most), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = big ? smem_bytes<64>(a.E) : smem_bytes<16>(a.E);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kKernels[big][a.swiglu ? 1 : 0], maps, p);
}

}  // namespace skinny
