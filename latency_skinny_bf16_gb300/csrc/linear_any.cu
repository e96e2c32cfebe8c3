// linear_any.cu -- products with an epilogue on CUDA cores, operands of any
// strides and alignment: Y[r][n] = epilogue(sum_c B(r, c) A(n, c)).
// Tiles of 64 x 64 outputs through shared memory, 4 x 4 a thread, rounded
// multiply-adds: right for every case, bound by the multiply-adds.
#include "act.cuh"
#include "common.cuh"
#include "experts_gemm.h"
#include "layer.h"

namespace skinny {
namespace {

constexpr int kT = 64, kC = 16, kThreads = 256;

__device__ __forceinline__ float element(const Operand &o, int64_t i, int64_t c) {
    return bf16_one(ldg_u16(o.p + (o.crossed ? c * o.ld + i : i * o.ld + c)));
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads) product_any_kernel(const __grid_constant__ ProductArgs p)
{
    constexpr int G = GATED ? 2 : 1;
    __shared__ float sa[G][kC][kT + 1], sb[kC][kT + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * kT;
    for (int64_t r0 = (int64_t)blockIdx.y * kT; r0 < p.rows; r0 += (int64_t)gridDim.y * kT) {
        float acc[G][4][4] = {};
        for (int c0 = 0; c0 < p.depth; c0 += kC) {
            for (int i = threadIdx.x; i < kT * kC; i += kThreads) {
                const int ca = p.A.crossed ? i / kT : i % kC, na = p.A.crossed ? i % kT : i / kC;
                const int cb = p.B.crossed ? i / kT : i % kC, nb = p.B.crossed ? i % kT : i / kC;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    sa[g][ca][na] = c0 + ca < p.depth && n0 + na < p.cols ? element(p.A, (int64_t)g * p.cols + n0 + na, c0 + ca) : 0.f;
                sb[cb][nb] = c0 + cb < p.depth && r0 + nb < p.rows ? element(p.B, r0 + nb, c0 + cb) : 0.f;
            }
            __syncthreads();
#pragma unroll 4
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[g][i][j] += sb[c][ty + 16 * i] * sa[g][c][tx + 16 * j];
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (r >= p.rows || n >= p.cols) continue;
                float z[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    z[g] = acc[g][i][j] + (p.bias ? bf16_one(p.bias[g * p.cols + n]) : 0.f);
                    if (p.Z) p.Z[r * p.ldz + g * p.cols + n] = f32_to_bf16_rn(z[g]);
                }
                float y = act_value(p.act, z[0]);
                if (GATED) y *= z[G - 1];
                if (p.R) y += p.out_bf16 ? bf16_one(ldg_u16(static_cast<const uint16_t *>(p.R) + r * p.ldr + n))
                                         : __ldcg(static_cast<const float *>(p.R) + r * p.ldr + n);
                store_y(p.Y, p.out_bf16, r * p.ldy + n, y);
            }
    }
}

}  // namespace

cudaError_t launch_product_any(const ProductArgs &a, const CallCtx &c, cudaStream_t stream) {
    ProductArgs p = a;
    void *args[] = {&p};
    const int64_t rt = (a.rows + kT - 1) / kT;
    return launch_plain(act_gated(a.act) ? (const void *)product_any_kernel<true> : (const void *)product_any_kernel<false>,
                        dim3((unsigned)((a.cols + kT - 1) / kT), (unsigned)(rt < 65535 ? rt : 65535)), kThreads, 0, stream,
                        c.pdl, args);
}

}  // namespace skinny
