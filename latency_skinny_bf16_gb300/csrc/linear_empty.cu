// linear_empty.cu -- a product with an epilogue over no depth: the sums are empty,
// and the epilogue (bias, activation, residual) is all there is to do.
#include "experts_gemm.h"
#include "product.cuh"

namespace skinny {
namespace {

constexpr int kThreads = 256;

template <bool GATED>
__global__ void __launch_bounds__(kThreads) linear_empty_kernel(const __grid_constant__ Epilogue e)
{
    follow();
    const int n = blockIdx.x * kThreads + threadIdx.x;
    if (n >= e.cols) return;
    for (int64_t r = blockIdx.y; r < e.rows; r += gridDim.y) {
        float z[1] = {e.bias ? bf16_one(ldg_u16(e.bias + n)) : 0.f};
        const float up = GATED && e.bias ? bf16_one(ldg_u16(e.bias + e.cols + n)) : 0.f;
        if (e.Z) {
            e.Z[r * e.ldz + n] = f32_to_bf16_rn(z[0]);
            if (GATED) e.Z[r * e.ldz + e.cols + n] = f32_to_bf16_rn(up);
        }
        act_rows(z, e.act);
        if (GATED) z[0] *= up;
        out_rows(e, z, r, n, 1);
    }
}

}  // namespace

cudaError_t launch_linear_empty(const ProductArgs &a, const CallCtx &c, cudaStream_t stream) {
    Epilogue e = epilogue_of(a);
    void *args[] = {&e};
    return launch_plain(act_gated(a.act) ? (const void *)linear_empty_kernel<true> : (const void *)linear_empty_kernel<false>,
                        dim3((unsigned)((a.cols + kThreads - 1) / kThreads), (unsigned)(a.rows < 4096 ? a.rows : 4096)),
                        kThreads, 0, stream, c.pdl, args);
}

}  // namespace skinny
