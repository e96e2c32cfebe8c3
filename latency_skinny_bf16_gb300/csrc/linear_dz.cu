// linear_dz.cu -- the elementwise part of a product's backward pass: dZ from dY
// and the kept Z, and the bias gradient, sums of dZ over the tokens.
//     dZ = dY act'(Z);  gated: dY U act'(G) for the gates, dY act(G) for the ups
// A stream through device memory (dY, Z, dZ once each); the exponentials take three
// fifths of the issue slots beside it (GB300: 8192 x 2 * 2048 SwiGLU 33 us, 5.0 TB/s;
// odd widths go element by element, six CTAs an SM: with its products 1001 x 1437
// 39.7 us, with three or eight 40.7 and 41.4).  A CTA takes 32 lanes of V columns
// and every eighth of its part of the tokens a row of threads; the bias gradient is
// summed along a thread's tokens, over the CTA's eight rows and then over the parts
// by a second kernel, in a fixed order.
// dZ is rounded to bf16 here, once, as the operand of both products: the tensor cores
// take no fp32, and a second bf16 term for what the rounding drops would double the depth
// of dX and the rows of dW (8192 tokens, 2 * 2048 x 7168: 250 us each as it is).  It puts
// both at 0.0023 of their norm from the definition, where their own rounding is 0.0017.
#include "act.cuh"
#include "common.cuh"
#include "experts_gemm.h"
#include "layer.h"

namespace skinny {
namespace {

constexpr int kRows = 8, kThreads = 32 * kRows;

template <int V>
struct Cols {
    uint16_t e[V];
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (V == 8) {
            const uint4 v = ldg_v4(p);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        } else {
            e[0] = ldg_u16(p);
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        if constexpr (V == 8) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (uint32_t)e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            p[0] = e[0];
        }
    }
};

template <int V, bool GATED, int ACT>      // ACT: 0 none, 1 SiLU, 2 GELU
__global__ void __launch_bounds__(kThreads, V == 8 ? 3 : 6) linear_dz_kernel(const __grid_constant__ LinearDzArgs p)
{
    constexpr int G = GATED ? 2 : 1, kBatch = 4;     // rows whose loads go out together
    if (p.beside) griddep_launch_dependents();
    else follow();
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int n = (blockIdx.x * 32 + lane) * V;
    const int64_t m0 = p.M * blockIdx.y / gridDim.y, m1 = p.M * (blockIdx.y + 1) / gridDim.y;
    float sum[G][V] = {};
    if (n < p.N) {
        for (int64_t mb = m0 + row; mb < m1; mb += kBatch * kRows) {
            Cols<V> dy[kBatch], z[kBatch][G];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t m = min(mb + k * kRows, m1 - 1);
                dy[k].load(p.dY + m * p.lddy + n);
                if constexpr (ACT != 0) {
#pragma unroll
                    for (int g = 0; g < G; ++g) z[k][g].load(p.Z + m * p.ldz + (int64_t)g * p.N + n);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t m = mb + k * kRows;
                if (m >= m1) break;
                Cols<V> o[G];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float d[G];
                    const float y = bf16_one(dy[k].e[i]);
                    d[0] = y;
                    if constexpr (ACT != 0) {
                        float a, da;
                        act_both<ACT == 2>(bf16_one(z[k][0].e[i]), a, da);
                        d[0] = y * da;
                        if constexpr (GATED) {
                            d[0] = y * bf16_one(z[k][G - 1].e[i]) * da;
                            d[G - 1] = y * a;
                        }
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        sum[g][i] = __fadd_rn(sum[g][i], d[g]);      // the same sum with and without dZ: never fused
                        o[g].e[i] = f32_to_bf16_rn(d[g]);
                    }
                }
                if (p.dZ) {
#pragma unroll
                    for (int g = 0; g < G; ++g) o[g].store(p.dZ + m * p.lddz + (int64_t)g * p.N + n);
                }
            }
        }
    }
    if (!p.dbias) {
        if (p.beside) griddep_wait();
        return;
    }
    __shared__ float part[kRows][32 * V];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) part[row][i * 32 + lane] = sum[g][i];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * V; i += kThreads) {
            const int at = blockIdx.x * 32 * V + i, from = i % V * 32 + i / V;
            if (at >= p.N) continue;
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kRows; ++q) v += part[q][from];
            p.partial[(int64_t)blockIdx.y * G * p.N + (int64_t)g * p.N + at] = v;
        }
    }
    if (p.beside) griddep_wait();
}

// out[i] = the parts' sums in order.
__global__ void __launch_bounds__(kThreads) sum_parts_kernel(const float *partial, int parts, int n, float *out)
{
    follow();
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
#pragma unroll 8
    for (int q = 0; q < parts; ++q) v += __ldcg(partial + (int64_t)q * n + i);
    out[i] = v;
}

template <int V>
const void *kernel_for(int act) {
    switch (act) {
        case SKINNY_ACT_SILU: return (const void *)linear_dz_kernel<V, false, 1>;
        case SKINNY_ACT_GELU: return (const void *)linear_dz_kernel<V, false, 2>;
        case SKINNY_ACT_SWIGLU: return (const void *)linear_dz_kernel<V, true, 1>;
        case SKINNY_ACT_GEGLU: return (const void *)linear_dz_kernel<V, true, 2>;
        default: return (const void *)linear_dz_kernel<V, false, 0>;
    }
}

}  // namespace

cudaError_t launch_linear_dz(const LinearDzArgs &a, const CallCtx &c, cudaStream_t stream) {
    const bool gated = act_gated(a.act);
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.dY) | reinterpret_cast<uintptr_t>(a.Z) | reinterpret_cast<uintptr_t>(a.dZ);
    const bool wide = bits % 16 == 0 && a.N % 8 == 0 && a.lddy % 8 == 0 && (!a.Z || a.ldz % 8 == 0) && (!a.dZ || a.lddz % 8 == 0);
    const int V = wide ? 8 : 1, rows = gated ? 2 * a.N : a.N;
    const int parts = dbias_parts(a.M);          // one part's sums are the bias gradient itself
    LinearDzArgs p = a;
    if (parts == 1) p.partial = a.dbias;
    void *args[] = {&p};
    const void *fn = wide ? kernel_for<8>(a.act) : kernel_for<1>(a.act);
    cudaError_t e = launch_plain(fn, dim3((unsigned)((a.N + 32 * V - 1) / (32 * V)), (unsigned)parts), kThreads, 0, stream, c.pdl, args);
    if (e != cudaSuccess || !a.dbias || parts == 1) return e;
    const float *partial = a.partial;
    int np = parts, n = rows;
    float *out = a.dbias;
    void *sargs[] = {&partial, &np, &n, &out};
    return launch_plain((const void *)sum_parts_kernel, dim3((unsigned)((rows + kThreads - 1) / kThreads)), kThreads, 0, stream, c.pdl, sargs);
}

}  // namespace skinny
