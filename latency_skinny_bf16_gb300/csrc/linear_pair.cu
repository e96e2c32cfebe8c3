// linear_pair.cu -- products with an epilogue on the fifth-generation tensor
// cores, for many rows: Y[r][n] = epilogue(sum_c B(r, c) A(n, c)).
//
// With many rows the tensor cores are the limit, and what feeds them: a pair of
// SMs works on one tile of 256 indexes of A by 256 rows of B (tcgen05.mma with
// cta_group::2), each SM holding half of A and half of B in shared memory and 128
// lanes x 256 columns of the sums in its tensor memory.  Against one SM's
// 128 x 256 that halves what shared memory and L2 deliver of B.
//   * Persistent: a cluster of two CTAs takes tiles in turn, eight tiles of rows
//     by every tile of A, so that what runs at a time shares its operands in L2.
//   * Warp 0 moves each CTA's boxes by tensor-map TMA into its ring, both CTAs'
//     copies of a stage completing on the first's barrier; the first's warp 1
//     issues the MMAs for both.  (The second telling the first when its own had
//     landed: 4864 x 4096 x 8192 at 1244 TFLOP/s.)  At most 64 MMAs are summed in tensor memory: two sets of 256 columns
//     in rotation, eight warps add each set into fp32 registers (128 rows of one
//     output each) while the tensor cores work on the other.  Reading a set holds
//     the tensor cores up, whatever it overlaps (4864 x 4096 x 8192:
//     181 us with 16 MMAs a set, 177 with 32, 174 with 64); 64 keep the bound of
//     the products, 64 * 2 * 2^-24 = 7.6e-6 of the terms' sum (measured: a third).
//   * At a tile's end these warps run the epilogue from their registers, and the
//     MMAs of the next tile go on for two sets.  With a gated activation a CTA's
//     lanes are 64 gates and their 64 ups; half of the rows of each change sides
//     through shared memory, so that all eight warps have the same work.
// What bounds it: the tensor cores, and each call's start and last tile.  GB300, us, in
// runs of 20 ms at 2070 MHz, and for seconds under the power limit (about 1440 MHz); in
// brackets the library's plain product:
//   4864 x 4096 x 8192                         171 [168], 200 [192]    1910 TFLOP/s, 1634
//   8192 rows SwiGLU 2048 x 7168, sums kept    260 [247], 303 [282]
//   its backward products                      248 [238] and 252 [243], 289 [271] and 293 [279]
//   2048 rows 7168 x 2048                      35 [33], 40 [37]; with bias and residual 41, 46
// Every wait is bounded; a CTA whose wait gave up reports it and stores nothing
// from there on, and both CTAs of a pair still meet at the end.
#include <cuda.h>

#include "experts_gemm.h"
#include "product.cuh"
#include "tma_stack.cuh"

namespace skinny {
namespace {

constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
constexpr uint64_t kLandNs = 2ull * 1000 * 1000;
enum : int { kWaitAcc = 5, kWaitAccEmpty = 6 };
constexpr int kDrainWarps = 8, kThreads = 64 + 32 * kDrainWarps;
constexpr int kHalf = 128 * 128;               // 128 indexes, 64 steps of the depth
constexpr int kStage = 2 * kHalf;              // of A and of B
constexpr int kSets = 2, kSetCols = 256;
constexpr int kChunk = 16;                     // stages summed in a set: 64 MMAs
constexpr int kBand = 8;                       // tiles of rows that run side by side
constexpr int kExchange = 2 * 16 * 1024;       // gated: two buffers
constexpr int kTail = 256;
__host__ __device__ constexpr int ring_stages(bool gated) { return gated ? 6 : 7; }
__host__ __device__ constexpr int smem_bytes(bool gated) {
    return 1024 + ring_stages(gated) * kStage + (gated ? kExchange : 0) + kTail;
}
static_assert(smem_bytes(false) <= kMaxDynSmem && smem_bytes(true) <= kMaxDynSmem, "shared memory");
// It takes all of tensor memory, so no other kernel's CTA that takes some may be on the SM.
static_assert(smem_bytes(true) + 1024 + kTcMinSmem + 1024 > 228 * 1024 && smem_bytes(false) + 1024 + kTcMinSmem + 1024 > 228 * 1024,
              "alone on an SM among kernels with tensor memory");

// ---- the pair's forms of tcgen05 and of the barriers between its CTAs
__device__ __forceinline__ void pair_alloc(uint32_t slot) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(slot), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(512) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrive on `bar` of both CTAs once every MMA issued so far has completed.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}
// A copy into this CTA that completes on a barrier of the pair's first CTA.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar) : "memory");
}
// The issuer waits for every stage, so all copies have landed once both CTAs meet at the end.  After a give-up
// some stages may never be complete on the barrier: a time in which any copy, and any arrival of a commit, lands.
__device__ __forceinline__ void let_land() {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kLandNs) {}
}

struct Maps {
    CUtensorMap a, b;
};
struct Params {
    Epilogue e;
    int nt, rt;          // tiles along A and along the rows
    int boxes;           // 64-step boxes of the depth
    int beside, last;
    int a3, b3;          // crossed operands by views [index / 64][step][64]: both boxes of a stage in one copy
    int *status;
    uint64_t budget_ns;
};

// Tile t: bands of kBand tiles of rows, the rows fastest.
__device__ __forceinline__ void tile_at(const Params &p, int64_t t, int &n, int &r) {
    const int64_t band = t / ((int64_t)kBand * p.nt);
    const int r0 = (int)band * kBand, high = min(kBand, p.rt - r0);
    const int in = (int)(t - band * kBand * p.nt);
    n = in / high;
    r = r0 + in % high;
}

template <bool GATED, bool AX, bool BX>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
linear_pair_kernel(const __grid_constant__ Maps maps, const Params p)
{
    constexpr int kStages = ring_stages(GATED);
    constexpr int TA = GATED ? 64 : 128;             // a CTA's outputs
    extern __shared__ uint8_t smem_raw[];
    if (p.beside && !p.last) griddep_launch_dependents();
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    float *exchange = reinterpret_cast<float *>(smem + kStages * kStage);
    constexpr int kBars = kStages * kStage + (GATED ? kExchange : 0);
    const uint32_t bars = base + kBars;
    auto full = [&](int s) { return bars + 8u * s; };                          // both CTAs' copies, on the first
    auto empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto accf = [&](int b) { return bars + 8u * (2 * kStages + b); };
    auto acce = [&](int b) { return bars + 8u * (2 * kStages + kSets + b); };  // both CTAs' warps, on the first
    const uint32_t done = bars + 8u * (2 * kStages + 2 * kSets);
    static_assert(8 * (2 * kStages + 2 * kSets + 1) + 16 <= kTail, "tail");
    uint8_t *tail = smem + kBars + 8 * (2 * kStages + 2 * kSets + 1);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int *mma_ok = reinterpret_cast<volatile int *>(tail + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_ctarank();
    const int64_t tiles = (int64_t)p.nt * p.rt, pairs = gridDim.x / 2, first = blockIdx.x / 2;
    if (tid == 0) {
        prefetch_tensormap(&maps.a);
        prefetch_tensormap(&maps.b);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < kSets; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 2 * kDrainWarps);
        }
        mbar_init(done, 1);
        *mma_ok = 0;
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        pair_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)));
        tc_fence_before();
    }
    __syncthreads();
    cluster_arrive_release();                        // both CTAs' barriers are there
    cluster_wait_acquire();
    tc_fence_after();
    if (!p.beside) follow();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---- TMA producer; the warp stays together and counts the ring's place, as the issuer.  An operand is one
        // copy a stage where its tensor map can say so (8192 x 4096 x 7168, both crossed: 303 us by one lane with two
        // copies each, 288 with one, 255 so).
        const bool one = elect_one();
        int s = 0;
        uint32_t phase = 1;                          // the ring is free at first
        bool go = true;
        for (int64_t t = first; go && t < tiles; t += pairs) {
            int tn, tr;
            tile_at(p, t, tn, tr);
            const int n0 = tn * 2 * TA + rank * TA, r0 = tr * 256 + rank * 128;
            for (int k = 0; k < p.boxes; ++k) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty(s), phase, p.budget_ns))) {
                    if (one) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitProducerEmpty);
                    go = false;
                    break;
                }
                const int c = k * 64;
                const uint32_t st = base + s * kStage, bar = mapa_shared(full(s), 0);
                if (one) {
                    if (rank == 0) mbar_arrive_expect_tx(full(s), (uint32_t)(2 * kStage));
                    if constexpr (AX) {
                        if (p.a3) {
                            pair_load_3d(st, &maps.a, 0, c, n0 / 64, bar);
                        } else {
                            pair_load_2d(st, &maps.a, n0, c, bar);
                            pair_load_2d(st + kBox, &maps.a, n0 + 64, c, bar);
                        }
                    } else if constexpr (GATED) {    // a stack of two: the gates' rows and the ups'
                        pair_load_3d(st, &maps.a, c, n0, 0, bar);
                    } else {
                        pair_load_2d(st, &maps.a, c, n0, bar);
                    }
                    if constexpr (BX) {
                        if (p.b3) {
                            pair_load_3d(st + kHalf, &maps.b, 0, c, r0 / 64, bar);
                        } else {
                            pair_load_2d(st + kHalf, &maps.b, r0, c, bar);
                            pair_load_2d(st + kHalf + kBox, &maps.b, r0 + 64, c, bar);
                        }
                    } else {
                        pair_load_2d(st + kHalf, &maps.b, c, r0, bar);
                    }
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // The MMAs' arrivals on `empty` come to both CTAs: all are here before this CTA may exit and leave its shared
        // memory to another.  The waits are those of the stages that would follow.
        for (int k = 0; go && k < kStages; ++k) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty(s), phase, p.budget_ns))) {
                if (one) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
                go = false;
            }
            if (++s == kStages) {
                s = 0;
                phase ^= 1;
            }
        }
        if (!go && one) let_land();
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- MMA issuer: the warp stays together, so that what the MMAs take is uniform, and the ring's
            // place is counted, not divided for (4864 x 4096 x 8192: 223 us by one lane with divisions, 185 so,
            // 174 with the producer's too)
            constexpr uint32_t idesc = product_idesc<256, 256, AX, BX>();
            constexpr uint64_t kStepA = AX ? 2048 >> 4 : 32 >> 4, kStepB = BX ? 2048 >> 4 : 32 >> 4;
            const uint64_t da = operand_desc<AX>(base, 0), db = operand_desc<BX>(base + kHalf, 0);
            const bool one = elect_one();
            int s = 0, b = 0;
            uint32_t phase = 0, free_phase = 1;      // of the ring's place and of the set; the sets are free at first
            bool go = true;
            for (int64_t t = first; go && t < tiles; t += pairs) {
                for (int k = 0; k < p.boxes; ++k) {
                    const bool starts = k % kChunk == 0;
                    if (starts && !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(acce(b), free_phase, p.budget_ns))) {
                        if (one) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAccEmpty);
                        go = false;
                        break;
                    }
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(full(s), phase, p.budget_ns))) {
                        if (one) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitConsumerFull);
                        go = false;
                        break;
                    }
                    tc_fence_after();
                    const bool ends = k % kChunk == kChunk - 1 || k == p.boxes - 1;
                    const uint64_t at = (uint64_t)(uint32_t)(s * (kStage >> 4));
                    if (one) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            pair_mma(tmem + (uint32_t)(b * kSetCols), da + at + j * kStepA, db + at + j * kStepB, idesc,
                                     !starts || j ? 1u : 0u);
                        pair_commit(empty(s));
                        if (ends) pair_commit(accf(b));
                    }
                    __syncwarp();
                    if (ends) {
                        b ^= 1;
                        if (b == 0) free_phase ^= 1;
                    }
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (one) {
                if (!go) let_land();
                pair_commit(done);
                if (mbar_wait_bounded(done, 0, kDrainNs)) {
                    *mma_ok = 1;
                    asm volatile("st.shared::cluster.u32 [%0], %1;"
                                 :: "r"(mapa_shared(smem_u32(const_cast<int *>(mma_ok)), 1)), "r"(1) : "memory");
                } else {
                    report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
                }
            }
        }
        __syncwarp();
    } else {
        // ---- draining warps: lane quarter q of tensor memory, half h of the columns
        const int q = warp & 3, h = (warp - 2) >> 2;
        const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(128 * h);
        const int chunks = (p.boxes + kChunk - 1) / kChunk;
        int64_t c = 0;
        bool ok = true;
        for (int64_t t = first; t < tiles; t += pairs) {
            int tn, tr;
            tile_at(p, t, tn, tr);
            if (p.e.R) {                                         // the residual's rows on their way to L2
                const int el = p.e.out_bf16 ? 2 : 4, n = GATED ? tn * 128 + rank * 64 + (32 * q & 63) : tn * 256 + rank * 128 + 32 * q;
                for (int j = lane; j < 128; j += 32)
                    if ((int64_t)tr * 256 + 128 * h + j < p.e.rows && n < p.e.cols)
                        prefetch_l2(static_cast<const char *>(p.e.R) + (((int64_t)tr * 256 + 128 * h + j) * p.e.ldr + n) * el);
            }
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            for (int k = 0; ok && k < chunks; ++k, ++c) {
                const int b = (int)(c % kSets);
                int got = 1;
                if (lane == 0) got = mbar_wait_bounded(accf(b), (uint32_t)((c / kSets) & 1), p.budget_ns);
                if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
                    if (lane == 0) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAcc);
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 128; j += 32) {
                    uint32_t r0[16], r1[16];
                    tmem_ld16_nowait(from + (uint32_t)(b * kSetCols + j), r0);
                    tmem_ld16_nowait(from + (uint32_t)(b * kSetCols + j + 16), r1);
                    tmem_ld_wait(r0);
                    tmem_ld_wait(r1);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        acc[j + i] += __uint_as_float(r0[i]);
                        acc[j + 16 + i] += __uint_as_float(r1[i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) remote_arrive(mapa_shared(acce(b), 0));
            }
            // ---- epilogue; a warp that gave up still meets the others at the exchange
            const Epilogue &e = p.e;
            const int row = 32 * q + lane;                       // of the CTA's 128
            const int64_t r0 = (int64_t)tr * 256 + 128 * h;
            const int rows = (int)max((int64_t)0, min((int64_t)128, e.rows - r0));
            if constexpr (!GATED) {
                const int n = tn * 256 + rank * 128 + row;
                if (ok && n < e.cols) {
                    if (e.bias) {
                        const float bias = bf16_one(ldg_u16(e.bias + n));
#pragma unroll
                        for (int j = 0; j < 128; ++j) acc[j] += bias;
                    }
                    if (e.Z) store_rows(acc, e.Z + r0 * e.ldz + n, e.ldz, rows);
                    act_rows(acc, e.act);
                    out_rows(e, acc, r0, n, rows);
                }
            } else {
                const bool up = q >= 2;
                const int l = row & 63, n = tn * 128 + rank * 64 + l;
                const bool live = ok && n < e.cols;
                const int jn = up ? e.cols + n : n;              // of the 2N sums
                if (live && e.bias) {
                    const float bias = bf16_one(ldg_u16(e.bias + jn));
#pragma unroll
                    for (int j = 0; j < 128; ++j) acc[j] += bias;
                }
                if (live && e.Z) store_rows(acc, e.Z + r0 * e.ldz + jn, e.ldz, rows);
                // gates keep rows 0 to 63 and get their ups, ups keep rows 64 to 127 and get their gates
                float y[64];
#pragma unroll
                for (int j = 0; j < 64; j += 16) {
                    float *buf = exchange + ((j >> 4) & 1) * 4096 + h * 2048;
#pragma unroll
                    for (int i = 0; i < 16; ++i) buf[(up ? 1024 : 0) + i * 64 + l] = up ? acc[j + i] : acc[64 + j + i];
                    __syncwarp();
                    named_bar_sync(2 + h, 128);
                    float g[16], u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float other = buf[(up ? 0 : 1024) + i * 64 + l];
                        g[i] = up ? other : acc[j + i];
                        u[i] = up ? acc[64 + j + i] : other;
                    }
                    act_rows(g, e.act);
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[j + i] = g[i] * u[i];
                }
                if (live) out_rows(e, y, r0 + (up ? 64 : 0), n, min(64, rows - (up ? 64 : 0)));
                __syncwarp();
                named_bar_sync(2 + h, 128);                      // the buffers are free for the next tile
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (p.beside) follow();
    cluster_arrive_release();                        // no thread of either CTA reads or signals the other from here on
    cluster_wait_acquire();
    if (warp == 1) {
        // the last commit's arrival, which the first CTA has seen in its own shared memory, in the second's
        if (rank == 1 && *mma_ok && !mbar_wait_bounded(done, 0, kDrainNs)) {
            if (lane == 0) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
        }
        __syncwarp();
        tc_fence_after();
        if (*mma_ok) pair_dealloc(tmem);
        // else an issued MMA may still write it: it stays allocated until the CTA exits
    }
}

template <bool GATED, bool AX, bool BX>
cudaError_t launch_as(const Maps &maps, const Params &p, int pairs, const CallCtx &c, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(GATED);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_pair_kernel<GATED, AX, BX>, maps, p);
}

}  // namespace

cudaError_t linear_pair_prepare() {
    cudaError_t e = set_max_dyn_smem(&linear_pair_kernel<false, false, false>);
    if (e == cudaSuccess) e = set_max_dyn_smem(&linear_pair_kernel<true, false, false>);
    if (e == cudaSuccess) e = set_max_dyn_smem(&linear_pair_kernel<false, true, false>);
    if (e == cudaSuccess) e = set_max_dyn_smem(&linear_pair_kernel<false, true, true>);
    return e;
}

// Up to 64 rows the tiles of 256 are mostly empty: 64 rows 24576 x 1536 22.6 us, and 15.2 with the depth split.
// Above, by the time of each: 0.276 us a box, 0.5 a tile and 4 a call.  GB300, us, this kernel and the other: 1024 rows
// 7168 x 2048 23.6 and 29.7, 2112 x 7168 35.6 and 30.9, 2048 x 2048 14.1 and 15.3; 192 rows 7168 x 2048 15.0 and 15.2;
// 128 rows 14.8 and 14.4; 512 rows 24576 x 1536 28.2 and 38.8, 384 rows 26.9 and 28.7 (where it takes the other).
bool linear_pair_faster(const ProductArgs &a, int num_sms) {
    if (a.rows <= 64 && !a.B.crossed) return false;
    const int64_t wide = act_gated(a.act) ? 128 : 256, pairs = num_sms / 2;
    const int64_t tiles = (a.rows + 255) / 256 * ((a.cols + wide - 1) / wide), boxes = depth_boxes(a.depth);
    return (tiles + pairs - 1) / pairs * (276 * boxes + 500) + 4000 < linear_tc_ns(a, num_sms);
}

cudaError_t launch_linear_pair(const ProductArgs &a, const CallCtx &c, cudaStream_t stream) {
    const bool gated = act_gated(a.act), ax = a.A.crossed, bx = a.B.crossed;
    const int TA = gated ? 64 : 128;
    const bool a3 = ax && a.cols % 64 == 0, b3 = bx && a.rows % 64 == 0;
    Maps maps;
    if (!(a3      ? encode_bf16_3d(&maps.a, a.A.p, a.cols, a.depth, a.A.ld, 64, 2)
          : ax    ? encode_bf16_2d(&maps.a, a.A.p, a.cols, a.depth, a.A.ld, 64)
          : gated ? encode_bf16_stack(&maps.a, a.A.p, a.depth, a.cols, 2, a.A.ld, a.A.ld * a.cols, 64, 2)
                  : encode_bf16_2d(&maps.a, a.A.p, a.depth, a.cols, a.A.ld, 128)) ||
        !(b3   ? encode_bf16_3d(&maps.b, a.B.p, (int)a.rows, a.depth, a.B.ld, 64, 2)
          : bx ? encode_bf16_2d(&maps.b, a.B.p, (int)a.rows, a.depth, a.B.ld, 64)
               : encode_bf16_2d(&maps.b, a.B.p, a.depth, (int)a.rows, a.B.ld, 128)))
        return cudaErrorInvalidValue;
    Params p{};
    p.e = epilogue_of(a);
    p.a3 = a3;
    p.b3 = b3;
    p.nt = (a.cols + 2 * TA - 1) / (2 * TA);
    p.rt = (int)((a.rows + 255) / 256);
    p.boxes = depth_boxes(a.depth);
    p.beside = a.beside;
    p.last = a.last;
    p.status = c.status;
    p.budget_ns = c.budget_ns;
    const int64_t tiles = (int64_t)p.nt * p.rt;
    const int pairs = (int)(tiles < c.num_sms / 2 ? tiles : c.num_sms / 2);
    if (ax) return bx ? launch_as<false, true, true>(maps, p, pairs, c, stream) : launch_as<false, true, false>(maps, p, pairs, c, stream);
    return gated ? launch_as<true, false, false>(maps, p, pairs, c, stream) : launch_as<false, false, false>(maps, p, pairs, c, stream);
}

}  // namespace skinny
