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
// of X at once; their sums are added in order through shared memory.  Per warp
// and step, 2 KB of W are in flight, so four CTAs on an SM cover device memory's
// latency.
// Rows of W that are not 16-byte aligned start at the same place within 16 bytes
// every P rows (P = 2, 4 or 8).  A tile is rows that do (kAlike): W comes in whole
// pieces as it lies, and X alone is shifted, by as many elements; the shifting is
// in registers.  (GB300, 16 rows, 60 experts 2816 x 4095: 79 us, 95 with W shifted
// too; 50 rows, 7 experts 7104 x 6333: 235 and 357, and 169 with two tiles of W to
// each shifted X, MT.)
// At most four MMAs (64 elements of K) are summed in the tensor core before a
// rounded add.
#include <type_traits>

#include "experts_gemm.h"
#include "mma_rows.cuh"

namespace skinny {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

enum Rows : int {
    kAny,                // of X and W; every piece of W is shifted too
    kAligned,            // 16 bytes
    kAlike,              // of X any, of W alike every P rows
};

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
    int P;               // kAlike
    Extent xe, we;
};

template <Rows ROWS, bool SWIGLU, int TT, int MT>
__global__ void __launch_bounds__(kThreads, TT == 1 ? 4 : 2)
experts_mma_kernel(const Params p)
{
    constexpr bool ALIGNED = ROWS == kAligned;
    extern __shared__ int smem[];
    __shared__ __align__(16) float part[kWarps][MT * TT][32][4];
    __shared__ int s_warp[kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int E = p.E, N = p.N;
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
    constexpr int kGroup = SWIGLU ? 8 : 16, kTileN = MT * kGroup;
    const int P = ROWS == kAlike ? p.P : 1;
    const int tiles = P * (((N + P - 1) / P + kTileN - 1) / kTileN);
    const int64_t line = (int64_t)found * tiles;
    const int KW = p.kw, kw = warp % KW, team = warp / KW, teams = kWarps / KW;
    auto meet = [&] {                                 // the warps of a team
        if (KW == 1) __syncwarp();
        else named_bar_sync(1 + team, 32 * KW);
    };
    for (int64_t i = (int64_t)blockIdx.x * teams + team; i < line; i += (int64_t)gridDim.x * teams) {
        const int a = (int)(i / tiles);
        const int in = (int)(i - (int64_t)a * tiles);
        const int e = active[a], c0 = in % P, j0 = in / P * kTileN;      // rows c0 + P j, j from j0 on
        const int J = (N - c0 + P - 1) / P;
        if (J <= 0) continue;
        const int r0 = row[e], r1 = row[e + 1];
        const uint16_t *We = p.W + (int64_t)e * p.ldwe;
        // rows past the end repeat the last one; they are not stored
        const uint16_t *wl[MT], *wh[MT];
#pragma unroll
        for (int i2 = 0; i2 < MT; ++i2) {
            const int j = j0 + i2 * kGroup + g;
            const int nl = c0 + P * min(j, J - 1), nh = SWIGLU ? N + nl : c0 + P * min(j + 8, J - 1);
            wl[i2] = We + (int64_t)nl * p.ldw;
            wh[i2] = We + (int64_t)nh * p.ldw;
        }
        // kAlike: the rows' elements are o behind the piece they start in
        const int o = ROWS == kAlike && p.K > 0 ? (int)(reinterpret_cast<uintptr_t>(wl[0]) & 15) / 2 : 0;
#pragma unroll
        for (int i2 = 0; i2 < MT; ++i2) {
            wl[i2] -= o;
            wh[i2] -= o;
        }
        const int K = p.K + o;
        for (int rb = r0; rb < r1; rb += 8 * TT) {
            const int nt = min(TT, (r1 - rb + 7) / 8);
            const uint16_t *x[TT];
            bool live[TT];
            bool inside = ROWS != kAny || (row_inside(wl[0], K, p.we) && row_inside(wh[0], K, p.we));
#pragma unroll
            for (int q = 0; q < TT; ++q) {
                live[q] = rb + 8 * q + g < r1;
                x[q] = p.X + (int64_t)(live[q] ? rb + 8 * q + g : rb) * p.ldx;
                if (!ALIGNED) inside = inside && row_inside(x[q], p.K, p.xe);
                x[q] -= o;
            }
            if (!ALIGNED) inside = __all_sync(0xFFFFFFFFu, inside);
            float acc[MT * TT][4];
#pragma unroll
            for (int q = 0; q < MT * TT; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[q][j] = 0.f;
            auto piece = [](const uint16_t *w) {
                if constexpr (ROWS == kAny) return load_whole8<false, true>(w, 0);
                // neighbours share sectors: through L1 where X leaves it room (GB300, 16 rows, 60 experts
                // 2816 x 4095: 79 us with, 82 without; 354 rows, 86 experts 318 x 6727: 282 and 190)
                if constexpr (ROWS == kAlike && TT == 1) return ldg16<true>(w);
                return ldg_stream_v4(w);
            };
            // the sums of the first NT token tiles
            auto sums = [&](auto NTc) {
                constexpr int NT = decltype(NTc)::value;
                auto products = [&](const uint4 (&l)[MT][2], const uint4 (&h)[MT][2], const uint4 (&v)[NT][2]) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int q = 0; q < NT; ++q) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_rows32(d, l[m][0], h[m][0], v[q][0]);
                            mma_rows32(d, l[m][1], h[m][1], v[q][1]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[m * TT + q][j] += d[j];
                        }
                };
                // the ends of the rows, or rows at an end of W or X
                auto ends = [&](int k) {
                    uint4 l[MT][2], h[MT][2], v[NT][2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int k8 = k + 32 * s + 8 * t;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            l[m][s] = load_row8<ROWS != kAny, true>(wl[m], k8, K, p.we, o);
                            h[m][s] = load_row8<ROWS != kAny, true>(wh[m], k8, K, p.we, o);
                        }
#pragma unroll
                        for (int q = 0; q < NT; ++q) {
                            v[q][s] = make_uint4(0, 0, 0, 0);
                            if (live[q]) v[q][s] = load_row8<ALIGNED, false>(x[q], k8, K, p.xe, o);
                        }
                    }
                    products(l, h, v);
                };
                int k = 64 * kw;
                if (ROWS == kAlike && k < o) {
                    ends(k);
                    k += 64 * KW;
                }
                if (inside) {
#pragma unroll MT == 1 ? 2 : 1
                    for (; k + 64 <= K; k += 64 * KW) {
                        uint4 l[MT][2], h[MT][2], v[NT][2];
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                l[m][s] = piece(wl[m] + k + 32 * s + 8 * t);
                                h[m][s] = piece(wh[m] + k + 32 * s + 8 * t);
                            }
#pragma unroll
                            for (int q = 0; q < NT; ++q) {
                                v[q][s] = make_uint4(0, 0, 0, 0);
                                if (live[q]) v[q][s] = load_whole8<ALIGNED, false>(x[q], k + 32 * s + 8 * t);
                            }
                        }
                        products(l, h, v);
                    }
                }
                for (; k < K; k += 64 * KW) ends(k);
            };
            if (TT == 1 || nt == 1) sums(std::integral_constant<int, 1>{});
            else if (nt == 2) sums(std::integral_constant<int, TT < 2 ? TT : 2>{});
            else sums(std::integral_constant<int, TT>{});
            // the results of 16 rows of W and token tile q from lane sl, its two rows of X
            auto result = [&](int m, int q, int sl, const float (&c)[4]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = rb + 8 * q + 2 * (sl & 3) + j, nj = j0 + m * kGroup + (sl >> 2);
                    if (r >= r1) continue;
                    const int64_t y = (int64_t)r * p.ldy + c0 + P * nj;
                    if constexpr (SWIGLU) {
                        if (nj < J) store_y(p.Y, p.out_bf16, y, c[j] / (1.f + expf(-c[j])) * c[2 + j]);
                    } else {
                        if (nj < J) store_y(p.Y, p.out_bf16, y, c[j]);
                        if (nj + 8 < J) store_y(p.Y, p.out_bf16, y + 8 * P, c[2 + j]);
                    }
                }
            };
            if (KW == 1) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int q = 0; q < TT; ++q)
                        if (q < nt) result(m, q, lane, acc[m * TT + q]);
                continue;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int q = 0; q < TT; ++q) {
                    const float (&c)[4] = acc[m * TT + q];
                    if (q < nt) *reinterpret_cast<float4 *>(part[warp][m * TT + q][lane]) = make_float4(c[0], c[1], c[2], c[3]);
                }
            meet();
            // the warps' sums in order
            for (int i2 = 32 * kw + lane; i2 < MT * nt * 32; i2 += 32 * KW) {
                const int m = MT == 1 ? 0 : (i2 >> 5) / nt, q = (i2 >> 5) - m * nt, sl = i2 & 31;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                for (int w = 0; w < KW; ++w) {
                    const float4 f = *reinterpret_cast<const float4 *>(part[team * KW + w][m * TT + q][sl]);
                    c[0] += f.x; c[1] += f.y; c[2] += f.z; c[3] += f.w;
                }
                result(m, q, sl, c);
            }
            meet();
        }
    }
}

template <Rows ROWS, bool SWIGLU, int TT, int MT>
cudaError_t launch_tt(const Params &p, int64_t tiles, const CallCtx &c, cudaStream_t stream) {
    Params q = p;
    void *args[] = {&q};
    const int64_t most = (TT == 1 ? 4 : 2) * (int64_t)c.num_sms, per = kWarps / p.kw, ctas = (tiles + per - 1) / per;
    return launch_plain((const void *)experts_mma_kernel<ROWS, SWIGLU, TT, MT>, dim3((unsigned)(ctas < most ? ctas : most)),
                        kThreads, 4 * (2 * p.E + 1), stream, c.pdl, args);
}
template <Rows ROWS, bool SWIGLU>
cudaError_t launch_as(const Params &p, int64_t tiles, bool many, bool pair, const CallCtx &c, cudaStream_t stream) {
    if (!many) return launch_tt<ROWS, SWIGLU, 1, 1>(p, tiles, c, stream);
    if constexpr (ROWS == kAlike) {
        if (pair) return launch_tt<ROWS, SWIGLU, 4, 2>(p, tiles, c, stream);
    }
    return launch_tt<ROWS, SWIGLU, 4, 1>(p, tiles, c, stream);
}

}  // namespace

cudaError_t launch_experts_mma(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream) {
    const uintptr_t xl = reinterpret_cast<uintptr_t>(a.X), wl = reinterpret_cast<uintptr_t>(a.W);
    const int64_t wrows = a.swiglu ? 2ll * a.N : a.N;
    const bool al = (xl | wl) % 16 == 0 && (a.ldx | a.ldw | a.ldwe) % 8 == 0;
    const int P = a.ldw % 8 == 0 ? 1 : a.ldw % 4 == 0 ? 2 : a.ldw % 2 == 0 ? 4 : 8;
    const bool alike = !al && (!a.swiglu || a.N % P == 0);   // an up lies as its gate
    const int per = a.swiglu ? 8 : 16, apart = alike ? P : 1;
    const int lines = ((a.N + apart - 1) / apart + per - 1) / per;      // tiles along N of one expert, of rows that lie alike
    const int64_t sets = (int64_t)(a.rows < a.E ? a.rows : a.E) * apart;
    // Rows of X held at once: 8, or 32 where the experts have more than 4 on average (GB300, 8 and 32 rows, us:
    // 256 experts 2048 x 2048, 1 row each 154 and 242; 8 experts 2048 x 2048, 16 rows each 34 and 24).  Where X is
    // shifted in registers and held 32 rows at a time, that is the work: two tiles of W share it while they still
    // give every CTA work (25 x 2 rows, 7 experts 7104 x 6333: 235 us, now 169; 8 experts 2 x 3712 x 6551, 49 rows
    // each: 914 and 636) and the last pair's empty half is little (86 experts 318 x 6727, three tiles: 193 and 220).
    const bool many = a.rows > 4 * a.E;
    const bool pair = many && alike && sets * lines >= 4ll * c.num_sms && (lines % 2 == 0 || lines >= 7);
    const int64_t tiles = sets * (pair ? (lines + 1) / 2 : lines);
    // Warps per tile: as many as K has pieces for on a long line; on a short one
    // the number with the least steps of K one after the other, rounds of tiles
    // times pieces of K per warp (the smaller number when equal: fewer sums to
    // join).  GB300, one token, 4 experts 2880 x 2880: 14.8 us with 4 warps a
    // tile (one round), 16.4 with 8 (two); 7 experts 208 x 5464: 13.5 and 8.4.
    const int pieces = (a.K + 63) / 64;
    const int64_t slots = (many ? 2ll : 4ll) * c.num_sms * kWarps;
    int kw = 1;
    int64_t best = -1;
    for (int w = 1; w <= kWarps && (w == 1 || w <= pieces); w *= 2) {
        const int64_t steps = ((tiles * w + slots - 1) / slots) * ((pieces + w - 1) / w);
        if (best < 0 || steps < best || tiles >= slots) { best = steps; kw = w; }
    }
    const Params p{a.X, a.ldx, a.rows, a.offsets, a.W, a.ldw, a.ldwe, a.E, a.N, a.K, a.out_bf16, a.Y, a.ldy,
                   kw, P, {xl, xl + (uintptr_t)(2 * ((a.rows - 1) * a.ldx + a.K))},
                   {wl, wl + (uintptr_t)(2 * ((a.E - 1) * a.ldwe + (wrows - 1) * a.ldw + a.K))}};
    if (al) return a.swiglu ? launch_as<kAligned, true>(p, tiles, many, pair, c, stream) : launch_as<kAligned, false>(p, tiles, many, pair, c, stream);
    if (!a.swiglu) return launch_as<kAlike, false>(p, tiles, many, pair, c, stream);
    return alike ? launch_as<kAlike, true>(p, tiles, many, pair, c, stream) : launch_as<kAny, true>(p, tiles, many, pair, c, stream);
}

}  // namespace skinny
