// heads.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and the gradients of both:
//     n = x / sqrt(mean x^2 + eps) w,  y = n turned by the token's angles
//     dx = r h - x r^3 mean(h x),  dw = sum g x r,   g = dy turned back, h = g w
// Every element is read once and written once: the kernels are a stream through
// device memory, and what they do beside it has to stay out of its way.
//   * L lanes hold a head (L a power of two), 32 / L heads a warp; a lane holds
//     chunks of V elements of both halves of the pairs, so that the rotation
//     stays within the lane and the only exchange is the sum over the L lanes.
//     V is the widest piece (16 bytes at most) that sizes, strides and pointers
//     allow.
//   * The angles of a token serve all of its heads: a warp takes one token and
//     walks its heads with cosines, sines and the norm's weight in registers,
//     kAhead steps of loads in flight.  With few tokens their heads are dealt to
//     more warps.
//   * The gradient of the weights is summed in registers over all that a warp
//     walks, then over the CTA's warps, then over the CTAs by a second kernel:
//     the order is fixed.
#include <type_traits>

#include "common.cuh"
#include "experts_gemm.h"
#include "layer.h"

namespace skinny {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPairs = 8;                    // pairs per lane at most

template <typename E, int V> struct RawOf;
template <> struct RawOf<uint16_t, 8> { using T = uint4; };
template <> struct RawOf<uint16_t, 4> { using T = uint2; };
template <> struct RawOf<uint16_t, 2> { using T = uint32_t; };
template <> struct RawOf<uint16_t, 1> { using T = unsigned short; };
template <> struct RawOf<float, 4> { using T = float4; };
template <> struct RawOf<float, 2> { using T = float2; };
template <> struct RawOf<float, 1> { using T = float; };

template <typename E, int V>
struct Piece {
    using Raw = typename RawOf<E, V>::T;
    union { Raw raw; E e[V]; };
    __device__ __forceinline__ void load(const E *p) { raw = __ldcg(reinterpret_cast<const Raw *>(p)); }
    __device__ __forceinline__ void load_shared(const E *p) { raw = __ldg(reinterpret_cast<const Raw *>(p)); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = E(0);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (std::is_same<E, float>::value) return e[i];
        else return bf16_one(e[i]);
    }
    __device__ __forceinline__ void set(int i, float v) {
        if constexpr (std::is_same<E, float>::value) e[i] = v;
        else e[i] = f32_to_bf16_rn(v);
    }
    __device__ __forceinline__ void store(E *p) const { *reinterpret_cast<Raw *>(p) = raw; }
};

struct Params {
    HeadsArgs a;
    int L;               // lanes per head
    int chunks, turned;  // chunks of a head, those that are turned
    int per, units;      // steps per unit, units per token
};

// Pairs (a[i], b[i]), or neighbours within a and within b, turned by the angles (back: turned back).
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float (&cs)[V], const float (&sn)[V], bool inter,
                                     bool back)
{
    const float f = back ? -1.f : 1.f;
    if (V > 1 && inter) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float c0 = cs[i], s0 = f * sn[i], c1 = cs[V / 2 + i], s1 = f * sn[V / 2 + i];
            const float u = a[2 * i], v = a[2 * i + 1], x = b[2 * i], y = b[2 * i + 1];
            a[2 * i] = u * c0 - v * s0;
            a[2 * i + 1] = v * c0 + u * s0;
            b[2 * i] = x * c1 - y * s1;
            b[2 * i + 1] = y * c1 + x * s1;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = a[i], v = b[i], s = f * sn[i];
            a[i] = u * cs[i] - v * s;
            b[i] = v * cs[i] + u * s;
        }
    }
}

template <typename E, int V, bool GRAD>
__global__ void __launch_bounds__(kThreads, 2) heads_kernel(const __grid_constant__ Params p)
{
    constexpr int NC = kPairs / V;           // chunks per lane
    constexpr int kAhead = GRAD ? 2 : 4;     // steps of loads in flight
    const HeadsArgs &a = p.a;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = p.L, sub = lane & (L - 1), hs = lane / L, HP = 32 / L;
    const int D = a.D, R = a.R, half = R / 2, rest = (D - R + 1) / 2;
    const bool inter = a.interleaved != 0;

    int ea[NC], eb[NC];                      // elements of the lane's chunks; -1: none
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = sub + L * j;
        ea[j] = eb[j] = -1;
        if (c < p.turned) {
            ea[j] = inter ? 2 * V * c : V * c;
            eb[j] = inter ? 2 * V * c + V : half + V * c;
        } else if (c < p.chunks) {
            ea[j] = R + V * (c - p.turned);
            eb[j] = ea[j] + rest;
            if (eb[j] >= D) eb[j] = -1;      // V == 1: the odd last element
        }
    }
    [[maybe_unused]] float dw[2][NC][2][V];
    if constexpr (GRAD) {
#pragma unroll
        for (int i = 0; i < 2 * NC * 2 * V; ++i) (&dw[0][0][0][0])[i] = 0.f;
    }
    auto over_head = [&](float v) {
        for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    };

    const int nq = (a.side[0].H + HP - 1) / HP, nk = (a.side[1].H + HP - 1) / HP, steps = nq + nk;
    const int64_t all = (int64_t)a.T * p.units;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < all; u += (int64_t)gridDim.x * kWarps) {
        const int t = (int)(u / p.units), s0 = (int)(u - (int64_t)t * p.units) * p.per, s1 = min(steps, s0 + p.per);
        float cs[NC][V], sn[NC][V];
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                cs[j][i] = 1.f;
                sn[j][i] = 0.f;
                const int c = sub + L * j;
                if (c < p.turned) {
                    const int pair = V * c + i, ax = a.pair_axis ? __ldg(a.pair_axis + pair) : 0;
                    const int at = ax >= 0 && ax < a.axes ? __ldg(a.positions + (int64_t)ax * a.T + t) : -1;
                    if (at >= 0 && at < a.P) {
                        const float *row = a.table + (int64_t)at * R + pair;
                        cs[j][i] = __ldg(row);
                        sn[j][i] = __ldg(row + half);
                    }
                }
            }
        auto walk = [&](auto SIDE, int b0, int b1) {
            constexpr int side = decltype(SIDE)::value;
            const HeadsSide &s = a.side[side];
            float w[NC][2][V];
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                Piece<E, V> pa, pb;
                pa.zero();
                pb.zero();
                const bool has = a.norm && s.w;
                if (has && ea[j] >= 0) pa.load_shared(static_cast<const E *>(s.w) + ea[j]);
                if (has && eb[j] >= 0) pb.load_shared(static_cast<const E *>(s.w) + eb[j]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    w[j][0][i] = has ? pa.get(i) : 1.f;
                    w[j][1][i] = has ? pb.get(i) : 1.f;
                }
            }
            for (int b = b0; b < b1; b += kAhead) {
                Piece<E, V> x[kAhead][NC][2];
                [[maybe_unused]] Piece<E, V> d[GRAD ? kAhead : 1][NC][2];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    const int h = (b + q) * HP + hs;
                    const bool live = b + q < b1 && h < s.H;
                    const E *xp = static_cast<const E *>(s.x) + (int64_t)t * s.st + (int64_t)h * s.sh;
                    [[maybe_unused]] const E *dp = static_cast<const E *>(s.d) + (int64_t)t * s.dst + (int64_t)h * s.dsh;
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        x[q][j][0].zero();
                        x[q][j][1].zero();
                        const bool need = live && (!GRAD || a.norm);
                        if (need && ea[j] >= 0) x[q][j][0].load(xp + ea[j]);
                        if (need && eb[j] >= 0) x[q][j][1].load(xp + eb[j]);
                        if constexpr (GRAD) {
                            d[q][j][0].zero();
                            d[q][j][1].zero();
                            if (live && ea[j] >= 0) d[q][j][0].load(dp + ea[j]);
                            if (live && eb[j] >= 0) d[q][j][1].load(dp + eb[j]);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    if (b + q >= b1) break;  // the whole warp
                    const int h = (b + q) * HP + hs;
                    float r = 1.f;
                    if (a.norm) {
                        float ss = 0.f;
#pragma unroll
                        for (int j = 0; j < NC; ++j)
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const float u0 = x[q][j][0].get(i), u1 = x[q][j][1].get(i);
                                ss += u0 * u0 + u1 * u1;
                            }
                        r = 1.f / sqrtf(over_head(ss) / (float)D + a.eps);
                    }
                    E *y = static_cast<E *>(s.y) + (int64_t)t * s.yst + (int64_t)h * s.ysh;
                    if constexpr (!GRAD) {
#pragma unroll
                        for (int j = 0; j < NC; ++j) {
                            float va[V], vb[V];
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                va[i] = x[q][j][0].get(i) * r * w[j][0][i];
                                vb[i] = x[q][j][1].get(i) * r * w[j][1][i];
                            }
                            if (R) turn<V>(va, vb, cs[j], sn[j], inter, false);
                            Piece<E, V> o;
#pragma unroll
                            for (int i = 0; i < V; ++i) o.set(i, va[i]);
                            if (h < s.H && ea[j] >= 0) o.store(y + ea[j]);
#pragma unroll
                            for (int i = 0; i < V; ++i) o.set(i, vb[i]);
                            if (h < s.H && eb[j] >= 0) o.store(y + eb[j]);
                        }
                    } else {
                        float ga[NC][V], gb[NC][V], hx = 0.f;
#pragma unroll
                        for (int j = 0; j < NC; ++j) {
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                ga[j][i] = d[q][j][0].get(i);
                                gb[j][i] = d[q][j][1].get(i);
                            }
                            if (R) turn<V>(ga[j], gb[j], cs[j], sn[j], inter, true);
                            if (a.norm) {
#pragma unroll
                                for (int i = 0; i < V; ++i) {
                                    const float xa = x[q][j][0].get(i), xb = x[q][j][1].get(i);
                                    if (h < s.H) {
                                        dw[side][j][0][i] += ga[j][i] * xa * r;
                                        dw[side][j][1][i] += gb[j][i] * xb * r;
                                    }
                                    ga[j][i] *= w[j][0][i];
                                    gb[j][i] *= w[j][1][i];
                                    hx += ga[j][i] * xa + gb[j][i] * xb;
                                }
                            }
                        }
                        float m = 0.f;
                        if (a.norm) m = r * r * r * (over_head(hx) / (float)D);
#pragma unroll
                        for (int j = 0; j < NC; ++j) {
                            Piece<E, V> o;
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                o.set(i, a.norm ? r * ga[j][i] - x[q][j][0].get(i) * m : ga[j][i]);
                            if (h < s.H && ea[j] >= 0) o.store(y + ea[j]);
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                o.set(i, a.norm ? r * gb[j][i] - x[q][j][1].get(i) * m : gb[j][i]);
                            if (h < s.H && eb[j] >= 0) o.store(y + eb[j]);
                        }
                    }
                }
            }
        };
        if (s0 < nq) walk(std::integral_constant<int, 0>{}, s0, min(s1, nq));
        if (s1 > nq) walk(std::integral_constant<int, 1>{}, max(s0, nq) - nq, s1 - nq);
    }

    if constexpr (GRAD) {
        if (!a.partial) return;
        __shared__ float part[kWarps][2][SKINNY_MAX_HEAD];
#pragma unroll
        for (int side = 0; side < 2; ++side)
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int ab = 0; ab < 2; ++ab)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float v = dw[side][j][ab][i];
                        for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
                        const int e = ab ? eb[j] : ea[j];
                        if (hs == 0 && e >= 0) part[warp][side][e + i] = v;
                    }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const int side = i >= D, e = i - side * D;
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) v += part[q][side][e];
            a.partial[((int64_t)blockIdx.x * 2 + side) * D + e] = v;
        }
    }
}

// The CTAs' sums, 32 elements a CTA: eight warps take every eighth part, then their sums in order.
__global__ void __launch_bounds__(kThreads) heads_weight_grad_kernel(const float *partial, int parts, int D, float *qw,
                                                                     float *kw)
{
    __shared__ float sum[kWarps][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (i < 2 * D)
#pragma unroll 8
        for (int q = warp; q < parts; q += kWarps) v += __ldcg(partial + (int64_t)q * 2 * D + i);
    sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && i < 2 * D) {
        for (int q = 1; q < kWarps; ++q) v += sum[q][lane];
        float *out = i < D ? qw : kw;
        if (out) out[i < D ? i : i - D] = v;
    }
}

// Whether pieces of `bytes` lie on their boundaries in every row of a side's tensor.
bool rows_lie(const void *p, int64_t st, int64_t sh, int el, int T, int H, int bytes) {
    uintptr_t bits = reinterpret_cast<uintptr_t>(p);
    if (T > 1) bits |= (uintptr_t)(st * el);
    if (H > 1) bits |= (uintptr_t)(sh * el);
    return bits % (uintptr_t)bytes == 0;
}

template <typename E, bool GRAD>
cudaError_t launch_as(const Params &p, int V, int ctas, cudaStream_t stream, bool pdl) {
    Params q = p;
    void *args[] = {&q};
    const void *fn;
    if constexpr (std::is_same<E, float>::value) {
        fn = V == 4 ? (const void *)heads_kernel<E, 4, GRAD> : V == 2 ? (const void *)heads_kernel<E, 2, GRAD>
                                                                      : (const void *)heads_kernel<E, 1, GRAD>;
    } else {
        fn = V == 8   ? (const void *)heads_kernel<E, 8, GRAD>
             : V == 4 ? (const void *)heads_kernel<E, 4, GRAD>
             : V == 2 ? (const void *)heads_kernel<E, 2, GRAD>
                      : (const void *)heads_kernel<E, 1, GRAD>;
    }
    return launch_plain(fn, dim3((unsigned)ctas), kThreads, 0, stream, pdl, args);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs &a, const CallCtx &c, cudaStream_t stream) {
    const int el = a.b16 ? 2 : 4;
    int V = 16 / el;
    for (; V > 1; V /= 2) {
        if (a.R / 2 % V || (a.D - a.R) % (2 * V)) continue;
        bool lie = true;
        for (const HeadsSide &s : a.side) {
            if (s.H == 0) continue;
            lie = lie && rows_lie(s.y, s.yst, s.ysh, el, a.T, s.H, V * el);
            if (!a.grad || a.norm) lie = lie && rows_lie(s.x, s.st, s.sh, el, a.T, s.H, V * el);
            if (a.grad) lie = lie && rows_lie(s.d, s.dst, s.dsh, el, a.T, s.H, V * el);
            if (a.norm && s.w) lie = lie && rows_lie(s.w, 0, 0, el, 1, 1, V * el);
        }
        if (lie) break;
    }
    Params p{};
    p.a = a;
    p.turned = a.R / 2 / V;
    p.chunks = p.turned + ((a.D - a.R + 1) / 2 + V - 1) / V;
    for (p.L = 1; p.L < p.chunks && p.L < 32;) p.L *= 2;
    const int HP = 32 / p.L, steps = (a.side[0].H + HP - 1) / HP + (a.side[1].H + HP - 1) / HP;
    // CTAs that an SM holds; a token's heads are dealt to more warps while there are fewer tokens than warps
    const int64_t ctas = 2ll * c.num_sms < kHeadsParts ? 2ll * c.num_sms : kHeadsParts, warps = ctas * kWarps;
    int64_t per = ((int64_t)a.T * steps + warps - 1) / warps;
    if (per > steps) per = steps;
    p.per = (int)per;
    p.units = (int)((steps + per - 1) / per);
    const int64_t need = ((int64_t)a.T * p.units + kWarps - 1) / kWarps;
    const int grid = (int)(need < ctas ? need : ctas);
    const bool sums = a.grad && (a.side[0].dw || a.side[1].dw);
    if (!sums) p.a.partial = nullptr;
    cudaError_t e = a.b16 ? (a.grad ? launch_as<uint16_t, true>(p, V, grid, stream, c.pdl) : launch_as<uint16_t, false>(p, V, grid, stream, c.pdl))
                          : (a.grad ? launch_as<float, true>(p, V, grid, stream, c.pdl) : launch_as<float, false>(p, V, grid, stream, c.pdl));
    if (e != cudaSuccess || !sums) return e;
    const float *partial = a.partial;
    int parts = grid, D = a.D;
    float *qw = a.side[0].dw, *kw = a.side[1].dw;
    void *args[] = {&partial, &parts, &D, &qw, &kw};
    return launch_plain((const void *)heads_weight_grad_kernel, dim3((unsigned)((2 * D + 31) / 32)), kThreads, 0, stream,
                        c.pdl, args);
}

}  // namespace skinny
