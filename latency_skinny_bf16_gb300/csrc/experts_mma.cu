// experts_mma.cu -- the experts' products with mma.sync, weights straight from
// device memory into its operands:
//     Y[r,n] = sum_k X[r,k] W[e][n][k]      offsets[e] <= r < offsets[e+1]
// or, with SwiGLU, g / (1 + exp(-g)) * u of the rows n and N + n of W[e].
// It serves weights and rows of any alignment, and the small calls where the
// tcgen05 kernel's long tiles leave SMs idle (the rule is at its launch).
//
// The 16-row tiles of W of the experts that have rows form one line (SwiGLU: 8
// gates on the MMA's rows 0..7, their ups on rows 8..15, so one thread ends up
// with both); the CTAs take its tiles in turn.  The eight warps of a CTA split
// K in pieces of 64 (or, in teams, fewer warps a tile), against up to 8 * TT rows
// of X at once; their sums are added in order through shared memory.  Per warp and step, 2 KB of W are in
// flight, so four CTAs on an SM cover device memory's latency.
// At most four MMAs (64 elements of K) are summed in the tensor core before a
// rounded add.
#include "experts_gemm.h"
#include "mma_rows.cuh"

namespace skinny {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Params {
    const uint16_t *X;
    int64_t ldx;
    int rows;
    const int32_t *offsets;
    const uint16_t *W;
    int64_t ldw, ldwe;
    int E, N, K;
    int out_bf16;
    void *Y;
    int64_t ldy;
    int kw;              // warps of a CTA along K: 1, 2, 4 or 8; its 8 / kw teams take tiles of their own
    Extent xe, we;
};

template <bool ALIGNED, bool SWIGLU, int TT>
__global__ void __launch_bounds__(kThreads, TT == 1 ? 4 : 2)
experts_mma_kernel(const Params p)
{
    extern __shared__ int smem[];
    __shared__ __align__(16) float part[kWarps][TT][32][4];
    __shared__ int s_warp[kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int E = p.E, N = p.N, K = p.K;
    int *row = smem;                                  // clamped offsets [E + 1]
    int *active = smem + E + 1;                       // the experts that have rows
    for (int e = tid; e <= E; e += kThreads)
        row[e] = p.offsets ? max(0, min(p.rows, __ldcg(p.offsets + e))) : e * p.rows;   // none: one matrix for all rows
    __syncthreads();
    int found = 0;
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = e0 + tid;
        const bool has = e < E && row[e + 1] > row[e];
        const unsigned ball = __ballot_sync(0xFFFFFFFFu, has);
        if (lane == 0) s_warp[warp] = __popc(ball);
        __syncthreads();
        int before = found;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_warp[w];
            found += s_warp[w];
        }
        if (has) active[before + __popc(ball & ((1u << lane) - 1))] = e;
        __syncthreads();
    }
    constexpr int kTileN = SWIGLU ? 8 : 16;
    const int tiles = (N + kTileN - 1) / kTileN;
    const int64_t line = (int64_t)found * tiles;
    const int KW = p.kw, kw = warp % KW, team = warp / KW, teams = kWarps / KW;
    auto meet = [&] {                                 // the warps of a team
        if (KW == 1) __syncwarp();
        else named_bar_sync(1 + team, 32 * KW);
    };
    for (int64_t i = (int64_t)blockIdx.x * teams + team; i < line; i += (int64_t)gridDim.x * teams) {
        const int a = (int)(i / tiles);
        const int e = active[a], n0 = (int)(i - (int64_t)a * tiles) * kTileN;
        const int r0 = row[e], r1 = row[e + 1];
        const uint16_t *We = p.W + (int64_t)e * p.ldwe;
        // rows past the end repeat the last one; they are not stored
        const int nl = min(n0 + g, N - 1), nh = SWIGLU ? N + nl : min(n0 + 8 + g, N - 1);
        const uint16_t *wl = We + (int64_t)nl * p.ldw, *wh = We + (int64_t)nh * p.ldw;
        for (int rb = r0; rb < r1; rb += 8 * TT) {
            const int nt = min(TT, (r1 - rb + 7) / 8);
            const uint16_t *x[TT];
            bool live[TT];
            bool inside = ALIGNED || (row_inside(wl, K, p.we) && row_inside(wh, K, p.we));
#pragma unroll
            for (int q = 0; q < TT; ++q) {
                live[q] = rb + 8 * q + g < r1;
                x[q] = p.X + (int64_t)(live[q] ? rb + 8 * q + g : rb) * p.ldx;
                if (!ALIGNED) inside = inside && row_inside(x[q], K, p.xe);
            }
            if (!ALIGNED) inside = __all_sync(0xFFFFFFFFu, inside);
            float acc[TT][4];
#pragma unroll
            for (int q = 0; q < TT; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[q][j] = 0.f;
            auto products = [&](const uint4 (&l)[2], const uint4 (&h)[2], const uint4 (&v)[TT][2]) {
#pragma unroll
                for (int q = 0; q < TT; ++q) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_rows32(d, l[0], h[0], v[q][0]);
                    mma_rows32(d, l[1], h[1], v[q][1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[q][j] += d[j];
                }
            };
            int k = 64 * kw;
            if (inside) {
#pragma unroll 2
                for (; k + 64 <= K; k += 64 * KW) {
                    uint4 l[2], h[2], v[TT][2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        l[s] = load_whole8<ALIGNED, true>(wl, k + 32 * s + 8 * t);
                        h[s] = load_whole8<ALIGNED, true>(wh, k + 32 * s + 8 * t);
#pragma unroll
                        for (int q = 0; q < TT; ++q) {
                            v[q][s] = make_uint4(0, 0, 0, 0);
                            if (live[q]) v[q][s] = load_whole8<ALIGNED, false>(x[q], k + 32 * s + 8 * t);
                        }
                    }
                    products(l, h, v);
                }
            }
            for (; k < K; k += 64 * KW) {             // the end of the rows, or rows at an end of W or X
                uint4 l[2], h[2], v[TT][2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    l[s] = load_row8<ALIGNED, true>(wl, k + 32 * s + 8 * t, K, p.we);
                    h[s] = load_row8<ALIGNED, true>(wh, k + 32 * s + 8 * t, K, p.we);
#pragma unroll
                    for (int q = 0; q < TT; ++q) {
                        v[q][s] = make_uint4(0, 0, 0, 0);
                        if (live[q]) v[q][s] = load_row8<ALIGNED, false>(x[q], k + 32 * s + 8 * t, K, p.xe);
                    }
                }
                products(l, h, v);
            }
            // the results of token tile q from lane sl, its two rows of X
            auto result = [&](int q, int sl, const float (&c)[4]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = rb + 8 * q + 2 * (sl & 3) + j, n = n0 + (sl >> 2);
                    if (r >= r1) continue;
                    const int64_t y = (int64_t)r * p.ldy + n;
                    if constexpr (SWIGLU) {
                        if (n < N) store_y(p.Y, p.out_bf16, y, c[j] / (1.f + expf(-c[j])) * c[2 + j]);
                    } else {
                        if (n < N) store_y(p.Y, p.out_bf16, y, c[j]);
                        if (n + 8 < N) store_y(p.Y, p.out_bf16, y + 8, c[2 + j]);
                    }
                }
            };
            if (KW == 1) {
#pragma unroll
                for (int q = 0; q < TT; ++q)
                    if (q < nt) result(q, lane, acc[q]);
                continue;
            }
#pragma unroll
            for (int q = 0; q < TT; ++q)
                if (q < nt) *reinterpret_cast<float4 *>(part[warp][q][lane]) = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
            meet();
            // the warps' sums in order
            for (int o = 32 * kw + lane; o < nt * 32; o += 32 * KW) {
                const int q = o >> 5, sl = o & 31;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                for (int w = 0; w < KW; ++w) {
                    const float4 f = *reinterpret_cast<const float4 *>(part[team * KW + w][q][sl]);
                    c[0] += f.x; c[1] += f.y; c[2] += f.z; c[3] += f.w;
                }
                result(q, sl, c);
            }
            meet();
        }
    }
}

template <bool ALIGNED, bool SWIGLU, int TT>
cudaError_t launch_tt(const Params &p, int64_t tiles, const CallCtx &c, cudaStream_t stream) {
    Params q = p;
    void *args[] = {&q};
    const int64_t most = (TT == 1 ? 4 : 2) * (int64_t)c.num_sms, per = kWarps / p.kw, ctas = (tiles + per - 1) / per;
    return launch_plain((const void *)experts_mma_kernel<ALIGNED, SWIGLU, TT>, dim3((unsigned)(ctas < most ? ctas : most)),
                        kThreads, 4 * (2 * p.E + 1), stream, c.pdl, args);
}
template <bool ALIGNED, bool SWIGLU>
cudaError_t launch_as(const Params &p, int64_t tiles, const CallCtx &c, cudaStream_t stream) {
    // rows of X held at once: 8, or 32 where the experts have more than 4 on average (GB300, TT 1 and 4, us:
    // 256 experts 2048 x 2048, 1 row each 154 and 242; 8 experts 2048 x 2048, 16 rows each 34 and 24)
    if (p.rows <= 4 * p.E) return launch_tt<ALIGNED, SWIGLU, 1>(p, tiles, c, stream);
    return launch_tt<ALIGNED, SWIGLU, 4>(p, tiles, c, stream);
}

}  // namespace

cudaError_t launch_experts_mma(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream) {
    const uintptr_t xl = reinterpret_cast<uintptr_t>(a.X), wl = reinterpret_cast<uintptr_t>(a.W);
    const int64_t wrows = a.swiglu ? 2ll * a.N : a.N;
    const int per = a.swiglu ? 8 : 16;
    const int64_t tiles = (int64_t)(a.rows < a.E ? a.rows : a.E) * ((a.N + per - 1) / per);
    // Warps per tile: as many as K has pieces for on a long line; on a short one
    // the number with the least steps of K one after the other, rounds of tiles
    // times pieces of K per warp (the smaller number when equal: fewer sums to
    // join).  GB300, one token, 4 experts 2880 x 2880: 14.8 us with 4 warps a
    // tile (one round), 16.4 with 8 (two); 7 experts 208 x 5464: 13.5 and 8.4.
    const int pieces = (a.K + 63) / 64;
    const int64_t slots = 4ll * c.num_sms * kWarps;
    int kw = 1;
    int64_t best = -1;
    for (int w = 1; w <= kWarps && (w == 1 || w <= pieces); w *= 2) {
        const int64_t steps = ((tiles * w + slots - 1) / slots) * ((pieces + w - 1) / w);
        if (best < 0 || steps < best || tiles >= slots) { best = steps; kw = w; }
    }
    const Params p{a.X, a.ldx, a.rows, a.offsets, a.W, a.ldw, a.ldwe, a.E, a.N, a.K, a.out_bf16, a.Y, a.ldy,
                   kw, {xl, xl + (uintptr_t)(2 * ((a.rows - 1) * a.ldx + a.K))},
                   {wl, wl + (uintptr_t)(2 * ((a.E - 1) * a.ldwe + (wrows - 1) * a.ldw + a.K))}};
    const bool al = (xl | wl) % 16 == 0 && (a.ldx | a.ldw | a.ldwe) % 8 == 0;
    if (al) return a.swiglu ? launch_as<true, true>(p, tiles, c, stream) : launch_as<true, false>(p, tiles, c, stream);
    return a.swiglu ? launch_as<false, true>(p, tiles, c, stream) : launch_as<false, false>(p, tiles, c, stream);
}

}  // namespace skinny
