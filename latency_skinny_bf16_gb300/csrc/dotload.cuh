// dotload.cuh -- eight bf16 elements of a row per lane at any alignment, for
// the CUDA-core dot products of the experts and the adapters.
#pragma once

#include "common.cuh"

namespace skinny {

// A warp covers 256 consecutive elements of a row from k0: with loads of V
// elements, lane l takes [k0 + u*32*V + l*V, +V) for u < 8 / V.  Elements from
// `len` on are zeros.  STREAM: read once, weights (non-allocating, read-only
// path); otherwise through L2 (the row may have just been written).
template <int V, bool STREAM>
__device__ __forceinline__ void load8(const uint16_t *row, int k0, int len, int lane, float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 8 / V; ++u) {
        const int k = k0 + u * 32 * V + lane * V;
        if (k + V <= len) {
            if constexpr (V == 8) {
                const uint4 q = STREAM ? ldg_stream_v4(row + k) : ldg_v4(row + k);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
            } else if constexpr (V == 4) {
                const uint2 q = STREAM ? ldg_stream_v2(row + k) : __ldcg(reinterpret_cast<const uint2 *>(row + k));
                v[4 * u] = bf16_lo(q.x); v[4 * u + 1] = bf16_hi(q.x);
                v[4 * u + 2] = bf16_lo(q.y); v[4 * u + 3] = bf16_hi(q.y);
            } else if constexpr (V == 2) {
                const uint32_t q = STREAM ? ldg_stream_u32(row + k) : __ldcg(reinterpret_cast<const uint32_t *>(row + k));
                v[2 * u] = bf16_lo(q); v[2 * u + 1] = bf16_hi(q);
            } else {
                v[u] = bf16_one(STREAM ? ldg_stream_u16(row + k) : ldg_u16(row + k));
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[V * u + i] = k + i < len ? bf16_one(ldg_u16(row + k + i)) : 0.f;
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

}  // namespace skinny
