// heads.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and the gradients of both:
//     n = x / sqrt(mean x^2 + eps) w,  y = n turned by the token's angles
//     dx = r h - x r^3 mean(h x),  dw = sum g x r,   g = dy turned back, h = g w
// Every element is read once and written once: the kernels are a stream through
// device memory, and what they do beside it has to stay out of its way.
//   * L lanes hold a head, 32 / L heads a warp; a lane holds chunks of V elements
//     of both halves of the pairs (or of neighbours), so that the rotation stays
//     within the lane and the only exchange is the sum over the L lanes.  V is the
//     widest piece (16 bytes at most) that sizes, strides and pointers allow.
//   * The angles of a token serve all of its heads: a warp walks an even share of
//     all heads, token by token, with the weights and the angles in registers as
//     the two factors that an element and its partner take, y = r (x p + partner q).
//   * The loads of the next steps are under way to shared memory (cp.async, each
//     thread's own slots, so no barrier) while one is computed, and the arithmetic
//     is in packed pairs of fp32.
//   * The gradient of the weights is summed in registers over all that a warp
//     walks, then over the CTA's warps, then over the CTAs by a second kernel:
//     the order is fixed.
// What bounds it: device memory nearly, for heads of whole 16-byte pieces, and the
// instructions (two thirds of the issue slots at 16 warps an SM, which is what the
// factors' registers leave).  GB300, bf16 heads of 128, 64 + 8 of them: 8192 tokens
// 55 us (5.5 TB/s), 16384 with three axes 108, the gradient for 8192 91 (5.0 TB/s);
// neighbours as pairs 55 and 93; fp32 32 + 8 heads 64 and 91.  Unusual sizes pay in
// instructions: 32 + 8 heads of 61 51 us (1.6 TB/s; the gradient 83), of 72 37, 16 + 2
// heads of 80 for 20000 tokens 50, 8 + 2 heads of 333 for 2048 tokens 26 (79).  Tried and
// slower: 24 warps of 80 registers (87 us where 16 take 59), two heads a lane at a
// time (the same), loads held in registers (60 against 55).
#include <type_traits>

#include "common.cuh"
#include "element_fetch.h"
#include "experts_gemm.h"
#include "layer.h"

namespace skinny {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPairs = 8;                    // pairs per lane at most

// ------------------------------------------------------------------ V values, two to a register pair
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <int V>
struct Vals {
    uint64_t p[V / 2];
    __device__ __forceinline__ void set(const float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) p[i] = pair2(v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) split2(p[i], v[2 * i], v[2 * i + 1]);
    }
};
template <>
struct Vals<1> {
    float p[1];
    __device__ __forceinline__ void set(const float (&v)[1]) { p[0] = v[0]; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = p[0]; }
};
template <int V>
__device__ __forceinline__ Vals<V> vfma(const Vals<V> &a, const Vals<V> &b, const Vals<V> &c) {
    Vals<V> r;
    if constexpr (V == 1) {
        r.p[0] = fmaf(a.p[0], b.p[0], c.p[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.p[i] = fma2(a.p[i], b.p[i], c.p[i]);
    }
    return r;
}
template <int V>
__device__ __forceinline__ Vals<V> vmul(const Vals<V> &a, const Vals<V> &b) {
    Vals<V> r;
    if constexpr (V == 1) {
        r.p[0] = a.p[0] * b.p[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.p[i] = mul2(a.p[i], b.p[i]);
    }
    return r;
}
template <int V>
__device__ __forceinline__ Vals<V> vall(float x) {
    Vals<V> r;
    if constexpr (V == 1) {
        r.p[0] = x;
    } else {
        const uint64_t two = pair2(x, x);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.p[i] = two;
    }
    return r;
}
template <int V>
__device__ __forceinline__ float vsum(const Vals<V> &a) {
    if constexpr (V == 1) {
        return a.p[0];
    } else {
        uint64_t s = a.p[0];
#pragma unroll
        for (int i = 1; i < V / 2; ++i) s = add2(s, a.p[i]);
        float lo, hi;
        split2(s, lo, hi);
        return lo + hi;
    }
}

// ------------------------------------------------------------------ V elements of memory
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
    static constexpr int kWords = sizeof(Raw) < 4 ? 1 : sizeof(Raw) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void put(const Raw &r) {
        if constexpr (sizeof(Raw) == 2) w[0] = r;
        else memcpy(w, &r, sizeof(Raw));
    }
    __device__ __forceinline__ void load(const E *p) { put(__ldcg(reinterpret_cast<const Raw *>(p))); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (std::is_same<E, float>::value) return __uint_as_float(w[i]);
        else return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
};
// The firsts and seconds of the pairs in a lane's two pieces: the pieces themselves, or, INTER, neighbours in both.
template <typename E, int V, bool INTER>
__device__ __forceinline__ void unpack(const Piece<E, V> &p, const Piece<E, V> &q, Vals<V> &a, Vals<V> &b) {
    float va[V], vb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (INTER) {
            const Piece<E, V> &from = 2 * i < V ? p : q;
            va[i] = from.at(2 * i % V);
            vb[i] = from.at(2 * i % V + 1);
        } else {
            va[i] = p.at(i);
            vb[i] = q.at(i);
        }
    }
    a.set(va);
    b.set(vb);
}
template <typename E, int V>
__device__ __forceinline__ void store_piece(E *p, const float (&v)[V]) {
    using Raw = typename RawOf<E, V>::T;
    Raw r;
    if constexpr (std::is_same<E, float>::value) {
        memcpy(&r, v, sizeof(Raw));
    } else if constexpr (V == 1) {
        r = f32_to_bf16_rn(v[0]);
    } else {
        uint32_t o[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        memcpy(&r, o, sizeof(Raw));
    }
    *reinterpret_cast<Raw *>(p) = r;
}
template <typename E, int V, bool INTER>
__device__ __forceinline__ void store_pair(E *y, int ea, int eb, const Vals<V> &a, const Vals<V> &b) {
    float va[V], vb[V];
    a.get(va);
    b.get(vb);
    if constexpr (INTER) {
        float p[V], q[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            (2 * i < V ? p : q)[2 * i % V] = va[i];
            (2 * i < V ? p : q)[2 * i % V + 1] = vb[i];
        }
        if (ea >= 0) store_piece<E, V>(y + ea, p);
        if (eb >= 0) store_piece<E, V>(y + eb, q);
    } else {
        if (ea >= 0) store_piece<E, V>(y + ea, va);
        if (eb >= 0) store_piece<E, V>(y + eb, vb);
    }
}

struct Params {
    HeadsArgs a;
    int L;               // lanes per head: 1 to 8, 16 or 32
    int chunks;          // of a head
    int together;        // entries of a table's row that lie on a boundary of their size: 4, 2 or 1
    float inv_d;
};

// 1 / sqrt(v): the approximation and a Newton step; 0 and infinity keep the approximation's.
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = rsqrtf(v);
    return v > 0.f && v < __int_as_float(0x7f800000) ? r * (1.5f - 0.5f * v * r * r) : r;
}

// Pieces of a step of heads under way to shared memory, each thread's own: kDepth steps of them.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__host__ __device__ constexpr int ring_depth(int el, bool grad) { return grad ? (el == 2 ? 3 : 2) : el == 2 ? 4 : 3; }
// A single bf16 element to the half of a slot that it has of its word in memory (element_fetch.h).
__device__ __forceinline__ void copy_element(uint32_t dst, const void *src, uintptr_t first, uintptr_t last) {
    const ElementFetch f = element_fetch(reinterpret_cast<uintptr_t>(src), first, last);
    if (f.bytes == 4) copy_async<4>(dst, reinterpret_cast<const void *>(f.from));
    else asm volatile("st.shared.u32 [%0], %1;" :: "r"(dst), "r"((uint32_t)ldg_u16(src) << (8 * (f.from & 2))) : "memory");
}
// Bytes of a thread's slot: a single bf16 element has a word.
__host__ __device__ constexpr int slot_bytes(int V, int el) { return V * el < 4 ? 4 : V * el; }
__host__ __device__ constexpr int chunks_per_lane(int V, bool wide) { return V > 1 ? kPairs / V : wide ? 8 : 2; }
__host__ __device__ constexpr int ring_bytes(int V, int NC, int el, bool grad) {
    return ring_depth(el, grad) * (grad ? 4 : 2) * NC * slot_bytes(V, el) * kThreads;
}

template <typename E, int V, int NC, bool GRAD, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) heads_kernel(const __grid_constant__ Params p)
{
    constexpr int kTensors = GRAD ? 2 : 1, kPieces = NC * 2 * kTensors, kBytes = slot_bytes(V, sizeof(E));
    constexpr int kDepth = ring_depth(sizeof(E), GRAD);
    constexpr bool kHalves = V * sizeof(E) < 4;      // slots hold an element and a neighbour
    static_assert(!INTER || V > 1, "neighbours in a piece");
    using Pc = Piece<E, V>;
    using Vs = Vals<V>;
    extern __shared__ __align__(16) uint8_t ring[];
    const HeadsArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = p.L, HP = 32 / L, hs = lane / L, sub = lane - hs * L;
    const int D = a.D, R = a.R, half = R / 2, rest = (D - R + 1) / 2, turned_chunks = half / V;
    // slots that no copy writes stay zero
    const uint32_t slots = smem_u32(ring) + threadIdx.x * kBytes;
    auto slot = [&](int stage, int piece) { return (stage * kPieces + piece) * kThreads * kBytes; };
    for (int i = 0; i < kDepth * kPieces; ++i)
#pragma unroll
        for (int k = 0; k < kBytes; k += 4) asm volatile("st.shared.u32 [%0], %1;" :: "r"(slots + slot(0, i) + k), "r"(0) : "memory");
    follow();

    // The lane's chunks: their two pieces' first elements (-1: none) and their pairs, by which the table is read.
    // Halves: elements i and R / 2 + i, then what is not turned in two halves.  INTER: neighbours, pieces c and
    // ceil(pieces / 2) + c of the head.
    const int second = (D / V + 1) / 2;
    int ea[NC], eb[NC];
    uint32_t axes[NC];                       // the axis of each of a chunk's pairs, four bits each; 15: not turned
    auto pair_of = [&](int c, int i) {
        if constexpr (INTER) return V * (i < V / 2 ? c : c + second) / 2 + i % (V / 2);
        else return c < turned_chunks ? V * c + i : half;
    };
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = sub + L * j;
        ea[j] = eb[j] = -1;
        axes[j] = 0xFFFFFFFFu;
        if (hs >= HP || c >= p.chunks) continue;
        if constexpr (INTER) {
            ea[j] = V * c;
            eb[j] = V * (c + second) < D ? V * (c + second) : -1;
        } else if (c < turned_chunks) {
            ea[j] = V == 1 && a.interleaved ? 2 * c : V * c;
            eb[j] = V == 1 && a.interleaved ? 2 * c + 1 : half + V * c;
        } else {
            ea[j] = R + V * (c - turned_chunks);
            eb[j] = ea[j] + rest;
            if (eb[j] >= D) eb[j] = -1;      // V == 1: the odd last element
        }
        axes[j] = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int pair = pair_of(c, i), ax = pair >= half ? -1 : a.pair_axis ? a.pair_axis[pair] : 0;
            axes[j] |= (uint32_t)(ax >= 0 && ax < a.axes ? ax : 15) << (4 * i);
        }
    }
    // the sum over a head's lanes, the same in each of them
    const bool pow2 = (L & (L - 1)) == 0;
    auto over_head = [&](float v) {
        if (pow2) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (o < L) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            return v;
        }
        float t = 0.f;
        for (int i = 0; i < L; ++i) t += __shfl_sync(0xFFFFFFFFu, v, hs * L + i);
        return t;
    };

    // The angles of token t: cosines and sines of the lane's pairs, and a bit for each pair that is not turned.
    // Positions and table may be what the preceding kernel writes: ordinary loads behind the wait, which see it, and
    // which neighbouring tokens' warps share in L1 (8192 tokens, 32 + 8 heads of 61: 48.6 us, past L1 51.5).  Never the
    // non-coherent path, whose memory has to be constant from the kernel's start on.
    constexpr int kRun = INTER ? V / 2 : V;                  // pairs that follow each other in the table
    auto angles = [&](int t, Vs (&cs)[NC], Vs (&sn)[NC]) {
        uint32_t still = 0;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float cv[V], sv[V];
            int at[V];                       // a pair's position; -1: not turned
            const int c = sub + L * j;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t ax = axes[j] >> (4 * i) & 15;
                if (i > 0 && ax == (axes[j] >> (4 * i - 4) & 15)) {
                    at[i] = at[i - 1];
                } else {
                    at[i] = ax < 15 ? a.positions[(int64_t)ax * a.T + t] : -1;
                    if (at[i] < 0 || at[i] >= a.P) at[i] = -1;
                }
                if (at[i] < 0) still |= 1u << (j * V + i);
            }
#pragma unroll
            for (int i = 0; i < V; i += kRun) {
                constexpr int kWide = kRun < 4 ? kRun : 4;
                bool one = kWide > 1 && p.together >= kWide && at[i] >= 0;
#pragma unroll
                for (int k = 1; k < kRun; ++k) one = one && at[i + k] == at[i];
                if (one) {
                    const float *row = a.table + (int64_t)at[i] * R + pair_of(c, i);
#pragma unroll
                    for (int k = 0; k < kRun; k += kWide) {
                        if constexpr (kWide == 4) {
                            const float4 c4 = *reinterpret_cast<const float4 *>(row + k);
                            const float4 s4 = *reinterpret_cast<const float4 *>(row + half + k);
                            cv[i + k] = c4.x; cv[i + k + 1] = c4.y; cv[i + k + 2] = c4.z; cv[i + k + 3] = c4.w;
                            sv[i + k] = s4.x; sv[i + k + 1] = s4.y; sv[i + k + 2] = s4.z; sv[i + k + 3] = s4.w;
                        } else if constexpr (kWide == 2) {
                            const float2 c2 = *reinterpret_cast<const float2 *>(row + k);
                            const float2 s2 = *reinterpret_cast<const float2 *>(row + half + k);
                            cv[i + k] = c2.x; cv[i + k + 1] = c2.y;
                            sv[i + k] = s2.x; sv[i + k + 1] = s2.y;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kRun; ++k) {
                        cv[i + k] = 1.f;
                        sv[i + k] = 0.f;
                        if (at[i + k] >= 0) {
                            const float *row = a.table + (int64_t)at[i + k] * R + pair_of(c, i + k);
                            cv[i + k] = row[0];
                            sv[i + k] = row[half];
                        }
                    }
                }
            }
            cs[j].set(cv);
            sn[j].set(sv);
        }
        return still;
    };

    [[maybe_unused]] Vs dw[NC][2];
    // Every warp has an even share of the queries' steps (a step is HP heads of a token) and of the keys', as they
    // follow each other in memory; the shares of the keys from the other end, for the calls with few.
    const int64_t warps = (int64_t)gridDim.x * kWarps, me = (int64_t)blockIdx.x * kWarps + warp;

    auto walk = [&](auto SIDE) {
        constexpr int side = decltype(SIDE)::value;
        const HeadsSide &s = a.side[side];
        const int steps = (s.H + HP - 1) / HP;
        const int64_t all = (int64_t)a.T * steps, mine = side ? warps - 1 - me : me;
        const int64_t begin = all * mine / warps, end = all * (mine + 1) / warps;
        if constexpr (GRAD) {
#pragma unroll
            for (int j = 0; j < NC; ++j) dw[j][0] = dw[j][1] = vall<V>(0.f);
        }
        if (begin == end) return;
        Pc wa[NC], wb[NC];                   // the norm's weight
        const bool weighted = a.norm && s.w;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            wa[j].zero();
            wb[j].zero();
            if (weighted && ea[j] >= 0) wa[j].load(static_cast<const E *>(s.w) + ea[j]);
            if (weighted && eb[j] >= 0) wb[j].load(static_cast<const E *>(s.w) + eb[j]);
        }
        int t = (int)(begin / steps), b = (int)(begin - (int64_t)t * steps), stage = 0;
        // the place of the step whose loads go out next, kDepth steps ahead of the one computed
        int64_t left = end - begin;
        int lt = t, lb = b;
        const E *lx, *ld = nullptr;
        const int64_t xstep = HP * s.sh, ystep = HP * s.ysh;
        [[maybe_unused]] const int64_t dstep = HP * s.dsh;
        auto load_token = [&] {
            lx = static_cast<const E *>(s.x) + (int64_t)lt * s.st + (int64_t)(lb * HP + hs) * s.sh;
            if constexpr (GRAD) ld = static_cast<const E *>(s.d) + (int64_t)lt * s.dst + (int64_t)(lb * HP + hs) * s.dsh;
        };
        load_token();
        // CAREFUL: the tensor's first or last heads, whose words may reach out of it
        auto issue = [&](int st, auto CAREFUL) {
            if (left > 0) {
                --left;
                const bool live = lb * HP + hs < s.H;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int q = i / (2 * NC), j = i / 2 % NC, at = i % 2 ? eb[j] : ea[j];
                    if (at < 0 || !live || (GRAD && q == 0 && !a.norm)) continue;
                    const E *from = (q ? ld : lx) + at;
                    const uint32_t dst = slots + slot(st, i);
                    if constexpr (decltype(CAREFUL)::value) {
                        const E *first = static_cast<const E *>(q ? s.d : s.x);
                        const E *last = first + (a.T - 1) * (q ? s.dst : s.st) + (s.H - 1) * (q ? s.dsh : s.sh) + D - 1;
                        copy_element(dst, from, reinterpret_cast<uintptr_t>(first), reinterpret_cast<uintptr_t>(last));
                    } else {
                        if constexpr (kHalves) from = reinterpret_cast<const E *>(reinterpret_cast<uintptr_t>(from) & ~(uintptr_t)3);
                        copy_async<kBytes>(dst, from);
                    }
                }
                lx += xstep;
                if constexpr (GRAD) ld += dstep;
                if (++lb == steps) {
                    lb = 0;
                    ++lt;
                    load_token();
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const int64_t careful = kHalves && end == all ? 1 : 0;       // steps at the share's end
        auto issue_next = [&](int st, bool starts) {
            if constexpr (kHalves) {
                if (left <= careful || (starts && begin == 0)) return issue(st, std::true_type{});
            }
            issue(st, std::false_type{});
        };
#pragma unroll
        for (int i = 0; i < kDepth; ++i) issue_next(i, i == 0);
        for (int64_t todo = end - begin; todo > 0; b = 0, ++t) {
            Vs cs[NC], sn[NC];
            const uint32_t still = angles(t, cs, sn);
            const bool some_still = __any_sync(0xFFFFFFFFu, still != 0);
            // factors of an element and of its partner, the weights among them (gradients: the angles themselves)
            [[maybe_unused]] Vs pa[NC], qa[NC], pb[NC], qb[NC];
            const Vs minus = vall<V>(-1.f);
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if constexpr (!GRAD) {
                    Vs va = vall<V>(1.f), vb = va;
                    if (weighted) unpack<E, V, INTER>(wa[j], wb[j], va, vb);
                    pa[j] = vmul(va, cs[j]);
                    qa[j] = vmul(vmul(vb, sn[j]), minus);
                    pb[j] = vmul(vb, cs[j]);
                    qb[j] = vmul(va, sn[j]);
                }
            }
            // v p + partner q; a pair that is not turned takes nothing of its partner, whatever that is
            auto turned = [&](int j, const Vs &va, const Vs &vb, Vs &oa, Vs &ob) {
                Vs ta = vb, tb = va;
                if (some_still) {
                    float fa[V], fb[V];
                    ta.get(fa);
                    tb.get(fb);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (still >> (j * V + i) & 1) fa[i] = fb[i] = 0.f;
                    ta.set(fa);
                    tb.set(fb);
                }
                if constexpr (!GRAD) {
                    oa = vfma(va, pa[j], vmul(ta, qa[j]));
                    ob = vfma(vb, pb[j], vmul(tb, qb[j]));
                } else {
                    oa = vfma(va, cs[j], vmul(ta, sn[j]));
                    ob = vfma(vmul(tb, sn[j]), minus, vmul(vb, cs[j]));
                }
            };
            int h = b * HP + hs;
            E *y = static_cast<E *>(s.y) + (int64_t)t * s.yst + (int64_t)h * s.ysh;
            for (; b < steps && todo > 0; ++b, --todo, h += HP, y += ystep) {
                asm volatile("cp.async.wait_group %0;" :: "n"(kDepth - 1) : "memory");
                Pc in[kTensors][NC][2];
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    Pc &to = in[i / (2 * NC)][i / 2 % NC][i % 2];
                    const uint32_t from = slots + slot(stage, i);
                    if constexpr (kBytes == 16)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(to.w[0]), "=r"(to.w[1]), "=r"(to.w[2]), "=r"(to.w[3]) : "r"(from) : "memory");
                    else if constexpr (kBytes == 8)
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(to.w[0]), "=r"(to.w[1]) : "r"(from) : "memory");
                    else
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(to.w[0]) : "r"(from) : "memory");
                    if constexpr (kHalves) {
                        // which half: the parity of the element's place
                        const bool d = i >= 2 * NC;
                        const uint32_t place = (uint32_t)(reinterpret_cast<uintptr_t>(d ? s.d : s.x) >> 1) +
                                               (uint32_t)t * (uint32_t)(d ? s.dst : s.st) + (uint32_t)h * (uint32_t)(d ? s.dsh : s.sh) +
                                               (uint32_t)(i % 2 ? eb[i / 2 % NC] : ea[i / 2 % NC]);
                        to.w[0] = to.w[0] >> (16 * (place & 1)) & 0xFFFFu;
                    }
                }
                issue_next(stage, false);
                if (++stage == kDepth) stage = 0;
                const bool live = hs < HP && h < s.H;
                Vs ss = vall<V>(0.f);
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    if (L * j >= p.chunks) break;
                    Vs xa, xb;
                    unpack<E, V, INTER>(in[0][j][0], in[0][j][1], xa, xb);
                    ss = vfma(xb, xb, vfma(xa, xa, ss));
                }
                const float r = a.norm ? inv_sqrt(fmaf(over_head(vsum(ss)), p.inv_d, a.eps)) : 1.f;
                const Vs rr = vall<V>(r);
                if constexpr (!GRAD) {
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        if (L * j >= p.chunks) break;
                        Vs xa, xb, oa, ob;
                        unpack<E, V, INTER>(in[0][j][0], in[0][j][1], xa, xb);
                        turned(j, xa, xb, oa, ob);
                        if (live) store_pair<E, V, INTER>(y, ea[j], eb[j], vmul(oa, rr), vmul(ob, rr));
                    }
                } else {
                    Vs ga[NC], gb[NC], hx = vall<V>(0.f);
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        if (L * j >= p.chunks) break;
                        Vs da, db, xa, xb;
                        unpack<E, V, INTER>(in[kTensors - 1][j][0], in[kTensors - 1][j][1], da, db);
                        turned(j, da, db, ga[j], gb[j]);
                        if (!a.norm) continue;
                        unpack<E, V, INTER>(in[0][j][0], in[0][j][1], xa, xb);
                        xa = vmul(xa, rr);                   // x r: its part of dw, and of the sum
                        xb = vmul(xb, rr);
                        if (live) {
                            dw[j][0] = vfma(ga[j], xa, dw[j][0]);
                            dw[j][1] = vfma(gb[j], xb, dw[j][1]);
                        }
                        if (weighted) {
                            Vs va, vb;
                            unpack<E, V, INTER>(wa[j], wb[j], va, vb);
                            ga[j] = vmul(ga[j], va);
                            gb[j] = vmul(gb[j], vb);
                        }
                        hx = vfma(ga[j], xa, vfma(gb[j], xb, hx));
                    }
                    // dx = r (h - x r mean(h x r))
                    const Vs c = vall<V>(a.norm ? -(r * (over_head(vsum(hx)) * p.inv_d)) : 0.f);
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        if (L * j >= p.chunks) break;
                        if (a.norm) {
                            Vs xa, xb;
                            unpack<E, V, INTER>(in[0][j][0], in[0][j][1], xa, xb);
                            ga[j] = vmul(vfma(xa, c, ga[j]), rr);
                            gb[j] = vmul(vfma(xb, c, gb[j]), rr);
                        }
                        if (live) store_pair<E, V, INTER>(y, ea[j], eb[j], ga[j], gb[j]);
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    };

    if constexpr (!GRAD) {
        walk(std::integral_constant<int, 0>{});
        walk(std::integral_constant<int, 1>{});
    } else {
        // every head's lanes by themselves: HP heads of D elements are no more than 32 lanes' pairs
        __shared__ float part[kWarps][2][32 * 2 * kPairs];
        auto keep = [&](int side) {
            if (!a.partial || hs >= HP) return;
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int ab = 0; ab < 2; ++ab) {
                    float all[V];
                    dw[j][ab].get(all);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        // INTER: pair i's first or second, in the piece that holds it
                        const int e = INTER ? (2 * i < V ? ea[j] : eb[j]) : ab ? eb[j] : ea[j];
                        const int k = INTER ? 2 * i % V + ab : i;
                        if (e >= 0) part[warp][side][hs * D + e + k] = all[i];
                    }
                }
        };
        walk(std::integral_constant<int, 0>{});
        keep(0);
        walk(std::integral_constant<int, 1>{});
        keep(1);
        if (!a.partial) return;
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const int side = i >= D, e = i - side * D;
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q)
                for (int g = 0; g < HP; ++g) v += part[q][side][g * D + e];
            if (gridDim.x > 1) a.partial[((int64_t)blockIdx.x * 2 + side) * D + e] = v;
            else if (a.side[side].dw) a.side[side].dw[e] = v;
        }
    }
}

// The CTAs' sums, 32 elements a CTA: its warps take the parts in turn, then their sums in order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) heads_weight_grad_kernel(const float *partial, int parts, int D, float *qw,
                                                                           float *kw)
{
    __shared__ float sum[kSumWarps][32];
    follow();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (i < 2 * D)
#pragma unroll 10
        for (int q = warp; q < parts; q += kSumWarps) v += __ldcg(partial + (int64_t)q * 2 * D + i);
    sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && i < 2 * D) {
        for (int q = 1; q < kSumWarps; ++q) v += sum[q][lane];
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

// wide: heads of more than 128 elements, where V == 1
template <typename E, bool GRAD>
const void *kernel_as(int V, bool wide, bool inter) {
    if constexpr (sizeof(E) == 2)
        if (V == 8) return inter ? (const void *)heads_kernel<E, 8, 1, GRAD, true> : (const void *)heads_kernel<E, 8, 1, GRAD, false>;
    if (V == 4) return inter ? (const void *)heads_kernel<E, 4, 2, GRAD, true> : (const void *)heads_kernel<E, 4, 2, GRAD, false>;
    if (V == 2) return inter ? (const void *)heads_kernel<E, 2, 4, GRAD, true> : (const void *)heads_kernel<E, 2, 4, GRAD, false>;
    return wide ? (const void *)heads_kernel<E, 1, 8, GRAD, false> : (const void *)heads_kernel<E, 1, 2, GRAD, false>;
}
const void *kernel_for(bool b16, int V, bool wide, bool grad, bool inter) {
    return b16 ? (grad ? kernel_as<uint16_t, true>(V, wide, inter) : kernel_as<uint16_t, false>(V, wide, inter))
               : (grad ? kernel_as<float, true>(V, wide, inter) : kernel_as<float, false>(V, wide, inter));
}

}  // namespace

cudaError_t heads_prepare() {
    for (int i = 0; i < 64; ++i) {
        const bool b16 = i & 1, grad = i & 2, inter = i & 4, wide = i & 8;
        const int V = 1 << (i >> 4);
        if (V == 8 && !b16) continue;
        const cudaError_t e = cudaFuncSetAttribute(kernel_for(b16, V, wide, grad, inter), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   ring_bytes(V, chunks_per_lane(V, wide), b16 ? 2 : 4, grad));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_heads(const HeadsArgs &a, const CallCtx &c, cudaStream_t stream) {
    const int el = a.b16 ? 2 : 4;
    int V = 16 / el;
    for (; V > 1; V /= 2) {
        if (a.interleaved ? a.D % V != 0 : a.R / 2 % V || (a.D - a.R) % (2 * V)) continue;
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
    const bool inter = a.interleaved && V > 1, wide = a.D > 128;
    p.chunks = inter ? (a.D / V + 1) / 2 : a.R / 2 / V + ((a.D - a.R + 1) / 2 + V - 1) / V;
    // the lanes per head that keep a warp's busiest: the fewest rounds of chunks for its heads, pieces of a head
    // that are 32 bytes together at least
    const int NC = chunks_per_lane(V, wide);
    p.L = 32;
    for (int L : {16, 8, 7, 6, 5, 4, 3, 2, 1}) {
        if (L * NC < p.chunks || (L * V * el < 32 && L < p.chunks)) continue;
        const int rounds = (p.chunks + L - 1) / L, best = (p.chunks + p.L - 1) / p.L;
        if (rounds * (32 / p.L) <= best * (32 / L)) p.L = L;
    }
    const uintptr_t table = reinterpret_cast<uintptr_t>(a.table);
    p.together = a.R % 8 == 0 && table % 16 == 0 ? 4 : a.R % 4 == 0 && table % 8 == 0 ? 2 : 1;
    p.inv_d = 1.f / (float)a.D;
    const int64_t ctas = 2ll * c.num_sms < kHeadsParts ? 2ll * c.num_sms : kHeadsParts;      // what an SM holds
    int64_t steps = 0;
    for (const HeadsSide &s : a.side) steps += (int64_t)a.T * ((s.H + 32 / p.L - 1) / (32 / p.L));
    const bool sums = a.grad && (a.side[0].dw || a.side[1].dw);
    const int64_t need = (steps + kWarps - 1) / kWarps;      // one CTA's sums are the weights' gradients themselves
    const int grid = (int)(need < ctas ? need : ctas);
    if (!sums) p.a.partial = nullptr;
    void *kargs[] = {&p};
    const cudaError_t e = launch_plain(kernel_for(a.b16, V, wide, a.grad, inter), dim3((unsigned)grid), kThreads,
                                       ring_bytes(V, NC, el, a.grad), stream, c.pdl, kargs);
    if (e != cudaSuccess || !sums || grid == 1) return e;
    const float *partial = a.partial;
    int parts = grid, D = a.D;
    float *qw = a.side[0].dw, *kw = a.side[1].dw;
    void *args[] = {&partial, &parts, &D, &qw, &kw};
    return launch_plain((const void *)heads_weight_grad_kernel, dim3((unsigned)((2 * D + 31) / 32)), 32 * kSumWarps, 0,
                        stream, c.pdl, args);
}

}  // namespace skinny
