// tma_stack.cuh -- tensor-map copies from a stack of matrices (tma.cuh has
// those of one matrix; the swizzle and the zeros outside are the same).
#pragma once

#include "tma.cuh"

namespace skinny {

// Box at (c0 = K element, c1 = row, c2 = matrix).
__device__ __forceinline__ void tma_load_stack(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                               uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}

// Host side (tmem_gemm.cu).  bf16 [n, rows, cols], row stride ld, matrix stride
// lde (elements), boxes of 64 columns x box_rows rows of one matrix.
bool encode_bf16_stack(CUtensorMap *map, const void *ptr, int cols, int64_t rows, int n, int64_t ld, int64_t lde,
                       int box_rows);

}  // namespace skinny
