// linear_tc.cu -- products with an epilogue on the fifth-generation tensor
// cores, for few rows: Y[r][n] = epilogue(sum_c B(r, c) A(n, c)).
//
// A's index is the MMA's M side (128 of a weight's rows; with a gated activation
// 64 gates and their 64 ups), up to BN rows of B its N side, so that the
// outputs' contiguous index lies along the lanes of tensor memory and A, the
// weight, is read once whatever the number of rows.
//   * A CTA has one tile and a slice of the depth: the S CTAs of a cluster split
//     it, so that small weights fill the GPU as well.  Two CTAs fit on an SM.
//   * Thread 0 moves 64-deep boxes of A and B by tensor-map TMA into a ring
//     (zeros outside), thread 32 issues tcgen05.mma into sets of tensor-memory
//     accumulators in rotation, at most 16 MMAs a set; warps 2 to 5 add each set
//     into fp32 registers.
//   * Both operands may lie crossed (the depth along the rows of memory), as the
//     backward pass needs them: the MMA reads either order.
//   * At the end every CTA sends each CTA of its cluster the partial sums of that
//     one's rows (BN / S of them), which it adds in the order of the CTAs before
//     the epilogue, neighbouring threads on neighbouring outputs.  One CTA for
//     the whole depth runs the epilogue from its registers.
// What bounds it: device memory for the weight, and, as far as calls follow each
// other, what lies between the preceding call's end and the first sums, and between
// the last sums and the stores (about 3 us).  GB300, us, chained with PDL, one token
// and 64, no bias: 2112 x 7168 8.1 and 10.4 (floor 4.5), 24576 x 1536 13.4 and 15.1 (11.3),
// SwiGLU 2048 x 7168 11.6 and 14.2 (8.8), 8192 x 8192 22.7 and 25.8 (20.0).
// Every wait is bounded; a CTA whose wait gave up reports it and stores nothing.
#include <cuda.h>
#include <type_traits>

#include "experts_gemm.h"
#include "product.cuh"
#include "tma.cuh"

namespace skinny {
namespace {

constexpr uint64_t kDrainNs = 200ull * 1000 * 1000;
enum : int { kWaitAcc = 5, kWaitAccEmpty = 6 };
constexpr int kThreads = 192;          // TMA warp, MMA warp, four draining warps
constexpr int kTmemCols = 256;
constexpr int kABytes = 128 * 128;     // 128 indexes of A, 64 steps of the depth

__host__ __device__ constexpr int stage_bytes(int BN) { return kABytes + BN * 128; }
__host__ __device__ constexpr int ring_stages(int BN) { return BN <= 16 ? 5 : BN <= 32 ? 4 : 3; }
__host__ __device__ constexpr int acc_sets(int BN) { return BN <= 64 ? 4 : 2; }
__host__ __device__ constexpr int set_cols(int BN) { return BN <= 64 ? 64 : BN; }
constexpr int kTail = 256;             // barriers, tensor-memory address, flags
// The partial sums that a CTA receives: 128 outputs by BN rows.  Up to 64 rows they have a place of their own, so that
// a CTA may send while others still sum; with 128 they take the ring's, once all of the cluster are done with theirs.
__host__ __device__ constexpr bool own_slots(int BN) { return BN <= 64; }
__host__ __device__ constexpr int slot_bytes(int BN) { return own_slots(BN) ? BN * 128 * 4 : 0; }
__host__ __device__ constexpr int smem_bytes(int BN) {
    return 1024 + ring_stages(BN) * stage_bytes(BN) + slot_bytes(BN) + kTail;
}
// tensor memory for two CTAs on an SM, as for every kernel that takes 256 columns of it
static_assert(smem_bytes(16) >= kTcMinSmem && smem_bytes(32) >= kTcMinSmem && smem_bytes(64) >= kTcMinSmem &&
              smem_bytes(128) >= kTcMinSmem && 2 * (smem_bytes(64) + 1024) <= 228 * 1024, "two CTAs on an SM");

struct Maps {
    CUtensorMap a, b;
};
struct Params {
    Epilogue e;
    int64_t mt;          // tiles along the rows of B
    int boxes;           // 64-step boxes of the depth
    int ta;              // outputs of a tile: 64 to 128 in steps of 8 (gated: 64)
    int split;           // CTAs of a cluster along the depth: 1, 2, 4 or 8
    int beside, last;
    int *status;
    uint64_t budget_ns;
};

template <int BN, bool GATED, bool AX, bool BX>
__global__ void __launch_bounds__(kThreads, 2) linear_tc_kernel(const __grid_constant__ Maps maps, const Params p)
{
    constexpr int kStages = ring_stages(BN), kStage = stage_bytes(BN), kSets = acc_sets(BN), kCols = set_cols(BN);
    constexpr int P = kCols / BN;                    // accumulators of a set, taken in turn: 4, 2 or 1
    const int TA = p.ta;
    static_assert(!BX || BN >= 64, "crossed boxes hold 64 indexes");
    extern __shared__ uint8_t smem_raw[];
    if (p.beside && !p.last) griddep_launch_dependents();
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    constexpr int kSlots = own_slots(BN) ? kStages * kStage : 0;       // where the partial sums arrive
    constexpr int kBars = kStages * kStage + slot_bytes(BN);
    const uint32_t bars = base + kBars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto accf = [&](int b) { return bars + 8u * (2 * kStages + b); };
    auto acce = [&](int b) { return bars + 8u * (2 * kStages + kSets + b); };
    const uint32_t done = bars + 8u * (2 * kStages + 2 * kSets);
    static_assert(8 * (2 * kStages + 2 * kSets + 1) + 16 <= kTail, "tail");
    uint8_t *tail = smem + kBars + 8 * (2 * kStages + 2 * kSets + 1);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
    volatile int *mma_ok = reinterpret_cast<volatile int *>(tail + 4);
    volatile int *failed = reinterpret_cast<volatile int *>(tail + 8);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.split, rank = S == 1 ? 0 : (int)cluster_ctarank();
    const int64_t tile = blockIdx.x / S;
    const int n0 = (int)(tile / p.mt) * TA;
    const int64_t r0 = tile % p.mt * BN;
    const int live = (int)min((int64_t)BN, p.e.rows - r0);
    const int b0 = (int)((int64_t)p.boxes * rank / S), nb = (int)((int64_t)p.boxes * (rank + 1) / S) - b0;
    auto load_a = [&](int i, int s) {
        const uint32_t st = base + s * kStage;
        const int c = (b0 + i) * 64;
        if constexpr (AX) {
            tma_load_2d(st, &maps.a, n0, c, full(s));
            tma_load_2d(st + kBox, &maps.a, n0 + 64, c, full(s));
        } else {
            tma_load_2d(st, &maps.a, c, n0, full(s));
            if (GATED) tma_load_2d(st + 64 * 128, &maps.a, c, p.e.cols + n0, full(s));
        }
    };
    const int tx = (AX ? kABytes : (GATED ? 2 : 1) * TA * 128) + BN * 128, pre = min(nb, kStages);
    if (tid == 0) {
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
        *failed = 0;
        fence_mbarrier_init_cluster();
        prefetch_tensormap(&maps.b);
        // A's first boxes, to L2 only: whatever the preceding kernel still writes, the copies behind the wait see it
        // (one token, 2112 x 7168 with a bias: 8.9 us without, 8.5 so, 8.4 with copies to shared memory here)
        for (int i = 0; !p.beside && i < pre; ++i) {
            const int c = (b0 + i) * 64;
            if constexpr (AX) {
                tma_prefetch_2d(&maps.a, n0, c);
                tma_prefetch_2d(&maps.a, n0 + 64, c);
            } else {
                tma_prefetch_2d(&maps.a, c, n0);
                if (GATED) tma_prefetch_2d(&maps.a, c, p.e.cols + n0);
            }
        }
    }
    if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (own_slots(BN) && S > 1) cluster_arrive_relaxed();              // this CTA is there to be sent to
    const uint32_t tmem = *tmem_slot;
    if (!p.beside) follow();

    float acc[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.f;
    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer
            auto load_b = [&](int i, int s) {
                const uint32_t st = base + s * kStage + kABytes;
                const int c = (b0 + i) * 64;
                if constexpr (BX) {
#pragma unroll
                    for (int j = 0; j < BN / 64; ++j) tma_load_2d(st + j * kBox, &maps.b, (int)r0 + 64 * j, c, full(s));
                } else {
                    tma_load_2d(st, &maps.b, c, (int)r0, full(s));
                }
            };
            for (int i = 0; i < pre; ++i) {
                mbar_arrive_expect_tx(full(i), (uint32_t)tx);
                load_a(i, i);
            }
            for (int i = 0; i < pre; ++i) load_b(i, i);
            int issued = pre;
            for (int i = pre; i < nb; ++i) {
                const int s = i % kStages;
                if (!mbar_wait_bounded(empty(s), (uint32_t)((i / kStages - 1) & 1), p.budget_ns)) {
                    report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitProducerEmpty);
                    break;
                }
                mbar_arrive_expect_tx(full(s), (uint32_t)tx);
                load_a(i, s);
                load_b(i, s);
                issued = i + 1;
            }
            // every copy issued has landed before the ring is used again or the CTA exits
            for (int i = max(0, issued - kStages); i < issued; ++i)
                if (!mbar_wait_bounded(full(i % kStages), (uint32_t)((i / kStages) & 1), kDrainNs)) {
                    report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
                    *failed = 1;
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer: the warp stays together, so that what the MMAs take is uniform
        constexpr uint32_t idesc = product_idesc<BN, 128, AX, BX>();
        constexpr uint64_t kStepA = AX ? 2048 >> 4 : 32 >> 4, kStepB = BX ? 2048 >> 4 : 32 >> 4;
        const uint64_t da = operand_desc<AX>(base, 0), db = operand_desc<BX>(base + kABytes, 0);
        const bool one = elect_one();
        int s = 0, b = 0;
        uint32_t phase = 0, free_phase = 1;          // of the ring's place and of the set; the sets are free at first
        for (int i = 0; i < nb; ++i) {
            const int in = i % 4;                    // stages of the set before this one
            if (in == 0 && !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(acce(b), free_phase, p.budget_ns))) {
                if (one) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAccEmpty);
                break;
            }
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(full(s), phase, p.budget_ns))) {
                if (one) report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitConsumerFull);
                break;
            }
            tc_fence_after();
            const bool ends = in == 3 || i == nb - 1;
            const uint64_t at = (uint64_t)(uint32_t)(s * (kStage >> 4));
            if (one) {
#pragma unroll
                for (int j = 0; j < 4; ++j)          // a stage's four MMAs go to the set's P accumulators in turn
                    umma_bf16(tmem + (uint32_t)(b * kCols + j % P * BN), da + at + j * kStepA, db + at + j * kStepB, idesc,
                              in == 0 && j < P ? 0u : 1u);
                umma_commit(empty(s));
                if (ends) umma_commit(accf(b));
            }
            __syncwarp();
            if (ends && ++b == kSets) {
                b = 0;
                free_phase ^= 1;
            }
            if (++s == kStages) {
                s = 0;
                phase ^= 1;
            }
        }
        if (one) {
            umma_commit(done);
            if (mbar_wait_bounded(done, 0, kDrainNs)) *mma_ok = 1;
            else report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitDrain);
        }
        __syncwarp();
    } else {
        // ---- draining warps: lane quarter warp % 4 of tensor memory
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int chunks = (nb + 3) / 4;
        for (int c = 0; c < chunks; ++c) {
            const int b = c % kSets;
            int got = 1;
            if (lane == 0) got = mbar_wait_bounded(accf(b), (uint32_t)((c / kSets) & 1), p.budget_ns);
            if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
                if (lane == 0) {
                    report_status(p.status, SKINNY_ERR_DEVICE_TIMEOUT, kWaitAcc);
                    *failed = 1;
                }
                break;
            }
            tc_fence_after();
            // the set's accumulators among each other first: one add to the long sum for 256 steps
#pragma unroll
            for (int j = 0; j < BN; j += 16) {
                uint32_t r[P][16];
#pragma unroll
                for (int q = 0; q < P; ++q) tmem_ld16_nowait(lanes + (uint32_t)(b * kCols + q * BN + j), r[q]);
#pragma unroll
                for (int q = 0; q < P; ++q) tmem_ld_wait(r[q]);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float v = __uint_as_float(r[0][i]);
                    if constexpr (P >= 2) v += __uint_as_float(r[1][i]);
                    if constexpr (P == 4) v += __uint_as_float(r[2][i]) + __uint_as_float(r[3][i]);
                    acc[j + i] += v;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce(b));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (*mma_ok) tmem_dealloc(tmem, kTmemCols);
        // else an issued MMA may still write it: it stays allocated until the CTA exits
    }

    // ---- partial sums to the rows' owners
    if (S > 1) {
        if (!own_slots(BN)) cluster_arrive_release();          // every CTA's ring has been read
        cluster_wait_acquire();                                // or: every CTA has started
    }
    const bool ok = *failed == 0 && *mma_ok != 0;
    const Epilogue &e = p.e;
    auto epilogue = [&] {
        if (!GATED && S == 1) {                          // from the registers: a thread has all rows of its output
            const int nl = 32 * (warp & 3) + lane, n = n0 + nl;
            if (warp >= 2 && ok && nl < TA && n < e.cols) {
                const float bias = e.bias ? bf16_one(ldg_u16(e.bias + n)) : 0.f;
#pragma unroll
                for (int j = 0; j < BN; ++j) acc[j] += bias;
                if (e.Z) store_rows(acc, e.Z + r0 * e.ldz + n, e.ldz, live);
                act_rows(acc, e.act);
                out_rows(e, acc, r0, n, live);
            }
            return;
        }
        const int shift = S == 1 ? 0 : S == 2 ? 1 : S == 4 ? 2 : 3, per = BN >> shift;      // rows of an owner
        // kVec rows of an output side by side, the outputs behind one another
        constexpr int kVec = BN < 32 ? 2 : 4;
        if (warp >= 2 && ok) {
            const uint32_t at = base + kSlots + 4u * (uint32_t)(rank * per * 128 + (32 * (warp & 3) + lane) * kVec);
            uint32_t to = at;
#pragma unroll
            for (int j = 0; j < BN; j += kVec) {
                if ((j & (per - 1)) == 0) to = mapa_shared(at, (uint32_t)(S == 1 ? rank : j / (BN / 8) >> (3 - shift)));
                if (j < live) {
                    if constexpr (kVec == 2)
                        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};"
                                     :: "r"(to), "f"(acc[j]), "f"(acc[j + 1]) : "memory");
                    else
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                                     :: "r"(to), "f"(acc[j]), "f"(acc[j + 1]), "f"(acc[j + 2]), "f"(acc[j + 3])
                                     : "memory");
                }
                to += 512u * kVec;
            }
        }
        if (S > 1) {
            cluster_arrive_release();
            cluster_wait_acquire();
        } else {
            __syncthreads();
        }
        if (!ok) return;
        // kRows rows of an output a thread at a time, the output's threads taking turns
        constexpr int kRows = BN < 8 ? BN : 8, kOuts = GATED ? 64 : 128, kTurns = kThreads / kOuts;
        const float *slots = reinterpret_cast<const float *>(smem + kSlots);
        const int nl = tid % kOuts, turn = tid / kOuts, n = n0 + nl, mine = min(per, live - rank * per);
        if (turn >= kTurns || nl >= TA || n >= e.cols) return;
        const float bias = e.bias ? bf16_one(ldg_u16(e.bias + n)) : 0.f;
        const float ubias = GATED && e.bias ? bf16_one(ldg_u16(e.bias + e.cols + n)) : 0.f;
        for (int c = turn * kRows; c < mine; c += kTurns * kRows) {
            const int rows = min(kRows, mine - c);
            float z[kRows], up[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) z[i] = up[i] = 0.f;
            for (int s = 0; s < S; ++s) {
                const float *slot = slots + (s * per + c) * 128 + nl * kVec;
#pragma unroll
                for (int i = 0; i < kRows; i += kVec) {
                    if (i >= rows) continue;
                    using Vec = typename std::conditional<kVec == 2, float2, float4>::type;
                    const Vec fz = *reinterpret_cast<const Vec *>(slot + i * 128);
                    const Vec fu = *reinterpret_cast<const Vec *>(slot + i * 128 + (GATED ? 64 * kVec : 0));
                    const float *v = reinterpret_cast<const float *>(&fz), *w = reinterpret_cast<const float *>(&fu);
#pragma unroll
                    for (int k = 0; k < kVec; ++k) {
                        z[i + k] += v[k];
                        if (GATED) up[i + k] += w[k];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                z[i] += bias;
                up[i] += ubias;
            }
            const int64_t r = r0 + rank * per + c;
            if (e.Z) {
                store_rows(z, e.Z + r * e.ldz + n, e.ldz, rows);
                if (GATED) store_rows(up, e.Z + r * e.ldz + e.cols + n, e.ldz, rows);
            }
            act_rows(z, e.act);
            if (GATED) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) z[i] *= up[i];
            }
            out_rows(e, z, r, n, rows);
        }
    };
    epilogue();
    if (p.beside) follow();
}

template <int BN, bool GATED, bool AX, bool BX>
cudaError_t launch_as(const Maps &maps, const Params &p, int64_t ctas, const CallCtx &c, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(BN);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_tc_kernel<BN, GATED, AX, BX>, maps, p);
}

template <int BN>
cudaError_t prepare_bn() {
    cudaError_t e = set_max_dyn_smem(&linear_tc_kernel<BN, false, false, false>);
    if (e == cudaSuccess) e = set_max_dyn_smem(&linear_tc_kernel<BN, true, false, false>);
    if (e == cudaSuccess) e = set_max_dyn_smem(&linear_tc_kernel<BN, false, true, false>);
    return e;
}

int rows_of_tile(const ProductArgs &a) {
    return a.B.crossed || a.rows > 64 ? 128 : a.rows > 32 ? 64 : a.rows > 16 ? 32 : 16;
}

// The depth over as many CTAs as the GPU holds clusters for, each with a set of MMAs at least; then tiles as low as
// make that many.  GB300, us, one token and 64: 24576 x 1536, 192 tiles of 128 and 280 of 88 14.5 and 13.9, 23 and
// 15; 7168 x 2048, four CTAs along the depth and two 9.7 and 9.6, 14.0 and 14.8; SwiGLU 2048 x 7168, eight and four
// 12.4 and 13.3, 16.2 and 17.4.  Of clusters of eight, 32 are at work at a time.
struct Split {
    int split, ta;
    int64_t ctas;
};
Split split_of(const ProductArgs &a, int BN, int num_sms) {
    const int full = act_gated(a.act) ? 64 : 128, boxes = depth_boxes(a.depth);
    const int64_t mt = (a.rows + BN - 1) / BN, across = mt * ((a.cols + full - 1) / full);
    const int64_t held[4] = {2ll * num_sms, 2ll * num_sms, 288ll * num_sms / 152, 256ll * num_sms / 152};
    int lg = 0;
    while (lg < 3 && across << (lg + 1) <= held[lg + 1] && boxes >= 4 << (lg + 1)) ++lg;
    Split s{1 << lg, full, 0};
    if (!a.A.crossed) {
        const int64_t most = (lg == 2 ? held[3] : held[lg]) / (s.split * mt);     // tiles along A
        int ta = full < 64 ? full : 64;
        while (ta < full && (a.cols + ta - 1) / ta > most) ta += 8;
        s.ta = ta;
    }
    s.ctas = mt * ((a.cols + s.ta - 1) / s.ta) * s.split;
    return s;
}

}  // namespace

// About the time of a call with more than 64 rows, in ns: two CTAs share an SM's tensor cores.  GB300, us, as
// measured and by this: 1024 rows 7168 x 2048 29.7 and 31.6, 24576 x 1536 73.7 and 75.6, 2112 x 7168 (two along the
// depth) 31.4 and 31.4, 512 rows SwiGLU 2048 x 7168 31.8 and 31.4, 2048 x 2048 (four) 13.4 and 12.2.
int64_t linear_tc_ns(const ProductArgs &a, int num_sms) {
    const Split s = split_of(a, 128, num_sms);
    const int64_t rounds = (s.ctas + 2 * num_sms - 1) / (2 * num_sms), boxes = (depth_boxes(a.depth) + s.split - 1) / s.split;
    return rounds * (400 * boxes + 3000) + (s.split > 1 ? 6000 : 0);
}

cudaError_t linear_tc_prepare() {
    cudaError_t e = prepare_bn<16>();
    if (e == cudaSuccess) e = prepare_bn<32>();
    if (e == cudaSuccess) e = prepare_bn<64>();
    if (e == cudaSuccess) e = prepare_bn<128>();
    if (e == cudaSuccess) e = set_max_dyn_smem(&linear_tc_kernel<128, false, true, true>);
    return e;
}

cudaError_t launch_linear_tc(const ProductArgs &a, const CallCtx &c, cudaStream_t stream) {
    const bool gated = act_gated(a.act), ax = a.A.crossed, bx = a.B.crossed;
    const int BN = rows_of_tile(a);
    Params p{};
    const Split plan = split_of(a, BN, c.num_sms);
    p.mt = (a.rows + BN - 1) / BN;
    p.boxes = depth_boxes(a.depth);
    p.split = plan.split;
    p.ta = plan.ta;
    const int TA = p.ta;
    Maps maps;
    const int arows = gated ? 2 * a.cols : a.cols;
    if (!(ax ? encode_bf16_2d(&maps.a, a.A.p, a.cols, a.depth, a.A.ld, 64)
             : encode_bf16_2d(&maps.a, a.A.p, a.depth, arows, a.A.ld, TA)) ||
        !(bx ? encode_bf16_2d(&maps.b, a.B.p, (int)a.rows, a.depth, a.B.ld, 64)
             : encode_bf16_2d(&maps.b, a.B.p, a.depth, (int)a.rows, a.B.ld, BN)))
        return cudaErrorInvalidValue;
    p.e = epilogue_of(a);
    p.beside = a.beside;
    p.last = a.last;
    p.status = c.status;
    p.budget_ns = c.budget_ns;
    const int64_t ctas = plan.ctas;
    if (ctas >= 1ll << 31) return cudaErrorInvalidValue;
#define SKINNY_TC(BNv)                                                              \
    case BNv:                                                                       \
        if (ax) return launch_as<BNv, false, true, false>(maps, p, ctas, c, stream); \
        return gated ? launch_as<BNv, true, false, false>(maps, p, ctas, c, stream) \
                     : launch_as<BNv, false, false, false>(maps, p, ctas, c, stream);
    if (bx) return launch_as<128, false, true, true>(maps, p, ctas, c, stream);
    switch (BN) {
        SKINNY_TC(16)
        SKINNY_TC(32)
        SKINNY_TC(64)
        SKINNY_TC(128)
    }
#undef SKINNY_TC
    return cudaErrorInvalidValue;
}

}  // namespace skinny
