// product.cuh -- what the products with an epilogue share on the fifth-
// generation tensor cores: operands of either order in shared memory, and the
// epilogue of one output.
#pragma once

#include "act.cuh"
#include "common.cuh"
#include "layer.h"
#include "tcgen05.cuh"

namespace skinny {

// A stage of an operand holds 64 steps of the depth in 128-byte swizzle atoms.
// Plain (depth along the 128-byte rows, sw128_desc): 16 steps further is 32
// bytes.  Crossed (the operand's index along the 128-byte rows): boxes of 64
// indexes x 64 steps, 8 KB each, one behind the other along the index; groups of
// 8 steps lie 1024 bytes apart, 16 steps further is 2048 bytes.
constexpr uint32_t kBox = 64 * 128;
__device__ __forceinline__ uint64_t crossed_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBox >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
template <bool CROSSED>
__device__ __forceinline__ uint64_t operand_desc(uint32_t stage, int step) {
    return CROSSED ? crossed_desc(stage + 2048u * step) : sw128_desc(stage + 32u * step);
}
// kind::f16 with operands of either order: bits 15 and 16 for a crossed A and B.
template <int N, int M, bool AX, bool BX>
__host__ __device__ constexpr uint32_t product_idesc() {
    return idesc_bf16<N, M>() | ((uint32_t)AX << 15) | ((uint32_t)BX << 16);
}

// One lane of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

struct Epilogue {
    const uint16_t *bias;
    const void *R;
    int64_t ldr;
    void *Y;
    int64_t ldy;
    uint16_t *Z;
    int64_t ldz;
    int64_t rows;
    int cols, act, out_bf16;
};
inline Epilogue epilogue_of(const ProductArgs &a) {
    return {a.bias, a.R, a.ldr, a.Y, a.ldy, a.Z, a.ldz, a.rows, a.cols, a.act, a.out_bf16};
}

// ---- the epilogue of N rows of one output, from registers.  Each step by itself, its types and pointers
// settled outside its loop, so that loads go out together and a row costs a step of a pointer.
template <typename T>
__device__ __forceinline__ uint32_t load_cg(const T *p) {     // a register each: halves of one would wait for each other
    if constexpr (sizeof(T) == 2) return ldg_u16(p);
    else return __float_as_uint(__ldcg(p));
}
// v[j] += R[j * ld], j < live
template <int N, typename T>
__device__ __forceinline__ void add_rows(float (&v)[N], const T *R, int64_t ld, int live) {
    if (live <= 0) return;
    constexpr int kBatch = N < 32 ? N : 32;
    const T *last = R + (live - 1) * ld;             // no branch around a load, so that they go out together
#pragma unroll
    for (int j = 0; j < N; j += kBatch) {
        uint32_t raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            raw[i] = load_cg(j + i < live ? R : last);
            R += ld;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[j + i] += __uint_as_float(sizeof(T) == 2 ? raw[i] << 16 : raw[i]);
    }
}
// Y[j * ld] = v[j], j < live; whole tiles without a row's predicate (64 rows' gradient of a 4096 x 7168 weight, 19.6 us,
// is 1 us longer with it)
template <int N, typename T>
__device__ __forceinline__ void store_rows(const float (&v)[N], T *Y, int64_t ld, int live) {
    auto put = [&](int j) {
        if constexpr (sizeof(T) == 2) *Y = f32_to_bf16_rn(v[j]);
        else *Y = v[j];
    };
    if (live >= N) {
#pragma unroll
        for (int j = 0; j < N; ++j, Y += ld) put(j);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j, Y += ld)
            if (j < live) put(j);
    }
}
template <int N>
__device__ __forceinline__ void act_rows(float (&v)[N], int act) {
    if (act == SKINNY_ACT_NONE) return;
    if (act_gelu(act)) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_value(SKINNY_ACT_GELU, v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_value(SKINNY_ACT_SILU, v[j]);
    }
}
// Residual and store of rows r .. r + live - 1 of output n.
template <int N>
__device__ __forceinline__ void out_rows(const Epilogue &e, float (&v)[N], int64_t r, int n, int live) {
    if (e.out_bf16) {
        if (e.R) add_rows(v, static_cast<const uint16_t *>(e.R) + r * e.ldr + n, e.ldr, live);
        store_rows(v, static_cast<uint16_t *>(e.Y) + r * e.ldy + n, e.ldy, live);
    } else {
        if (e.R) add_rows(v, static_cast<const float *>(e.R) + r * e.ldr + n, e.ldr, live);
        store_rows(v, static_cast<float *>(e.Y) + r * e.ldy + n, e.ldy, live);
    }
}

}  // namespace skinny
