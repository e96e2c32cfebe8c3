// mma_rows.cuh -- rows of a weight straight from device memory into mma.sync
// operands, for products with a few rows of X: no shared memory, no barrier,
// every load 16 bytes, at any alignment of the rows.
//
// mma.m16n8k16 sums over 16 k slots; which element of K sits in which slot is
// free as long as both operands agree.  Lane (g = lane / 4, t = lane % 4) holds
// slots 2t, 2t+1, 2t+8, 2t+9 of weight rows g and g + 8 and of token g.  So for
// 32 consecutive elements from k0 a lane loads the 8 elements from k0 + 8t of
// each of its three rows (16 bytes), the first four feeding one MMA, the other
// four a second:  element 8t + 4i + {0,1} -> slots 2t, 2t+1 of MMA i,
//                 element 8t + 4i + {2,3} -> slots 2t+8, 2t+9.
// The result's lane holds weight row g (c[0], c[1]) and g + 8 (c[2], c[3]) for
// tokens 2t and 2t + 1.
#pragma once

#include "common.cuh"

namespace skinny {

// A matrix (or a stack of them) as loads may touch it: the first element and
// the end of the last row.  An unaligned row is read in whole 16-byte pieces
// while these lie inside; they hold neighbouring rows' elements, cut off below.
struct Extent {
    uintptr_t lo, hi;
};

template <bool STREAM>
__device__ __forceinline__ uint4 ldg16(const void *p) {
    // STREAM: a weight, read-only; cached in L1 when unaligned neighbours share pieces
    if constexpr (STREAM) return __ldg(reinterpret_cast<const uint4 *>(p));
    return ldg_v4(p);
}

// The 16 bytes from byte `off` (even) of the 32 of q and r.
__device__ __forceinline__ uint4 shifted16(const uint4 &q, const uint4 &r, int off) {
    uint32_t w0 = q.x, w1 = q.y, w2 = q.z, w3 = q.w, w4 = r.x, w5 = r.y, w6 = r.z, w7 = r.w;
    if (off & 8) { w0 = w2; w1 = w3; w2 = w4; w3 = w5; w4 = w6; w5 = w7; }
    if (off & 4) { w0 = w1; w1 = w2; w2 = w3; w3 = w4; w4 = w5; }
    if (off & 2) {
        w0 = __funnelshift_r(w0, w1, 16);
        w1 = __funnelshift_r(w1, w2, 16);
        w2 = __funnelshift_r(w2, w3, 16);
        w3 = __funnelshift_r(w3, w4, 16);
    }
    return make_uint4(w0, w1, w2, w3);
}

// Whether every whole 16-byte piece that holds an element of row[0, len) lies inside the extent.
__device__ __forceinline__ bool row_inside(const uint16_t *row, int len, const Extent &ext) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row);
    return (a & ~(uintptr_t)15) >= ext.lo && ((a + 2 * (uintptr_t)len + 15) & ~(uintptr_t)15) <= ext.hi;
}

// Eight bf16 elements from element k of `row`, all below its length; not
// ALIGNED: the row is inside its extent (row_inside).  No branch, so loads batch.
template <bool ALIGNED, bool STREAM>
__device__ __forceinline__ uint4 load_whole8(const uint16_t *row, int k) {
    const uint16_t *at = row + k;
    if constexpr (ALIGNED) {
        return STREAM ? ldg_stream_v4(at) : ldg_v4(at);
    } else {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), a0 = a & ~(uintptr_t)15;
        const int off = (int)(a - a0);
        // an aligned row reads its one piece twice rather than the piece behind it
        const uint4 q = ldg16<STREAM>(reinterpret_cast<const void *>(a0));
        const uint4 r = ldg16<STREAM>(reinterpret_cast<const void *>(a0 + (off ? 16 : 0)));
        return shifted16(q, r, off);
    }
}

// Eight bf16 elements from element k of `row`, those before `first` and from
// `len` on zero: ends of rows, and rows at the ends of their extent.
template <bool ALIGNED, bool STREAM>
__device__ __forceinline__ uint4 load_row8(const uint16_t *row, int k, int len, const Extent &ext, int first = 0) {
    const uint16_t *at = row + k;
    if constexpr (ALIGNED) {
        if (k >= first && k + 8 <= len) return STREAM ? ldg_stream_v4(at) : ldg_v4(at);
    } else {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), a0 = a & ~(uintptr_t)15;
        const int off = (int)(a - a0);
        if (k >= first && k + 8 <= len && a0 >= ext.lo && a0 + (off ? 32 : 16) <= ext.hi)
            return load_whole8<ALIGNED, STREAM>(row, k);
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (k + e >= first && k + e < len) w[e >> 1] |= (uint32_t)ldg_u16(at + e) << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// c += rows . x^T over the 32 elements of one load_row8 per operand.
__device__ __forceinline__ void mma_rows32(float (&c)[4], const uint4 &lo, const uint4 &hi, const uint4 &x) {
    const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
    mma_bf16_16816(c, a0, x.x, x.y, c);
    mma_bf16_16816(c, a1, x.z, x.w, c);
}

}  // namespace skinny
