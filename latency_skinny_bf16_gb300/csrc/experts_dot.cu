// experts_dot.cu -- the experts' products on CUDA cores, for weights and rows
// of any alignment:
//     Y[r,n] = sum_k X[r,k] W[e][n][k]      offsets[e] <= r < offsets[e+1]
// or, with SwiGLU, g / (1 + exp(-g)) * u of the rows n and N + n of W[e].
//
// Grid (blocks of W rows, E): a CTA of an expert without rows leaves at once.
// A warp holds four rows of W (SwiGLU: two gates and their ups) against eight
// rows of X: per 256 elements of K every lane loads 8 elements of each, so W,
// which bounds it, is read once per eight rows of X.  Each lane sums its 8
// products in order, adds that to its running sum, and the warp adds its lanes
// in a butterfly: the longest chain of rounded adds is 8 + K / 256 + 5.
#include "dotload.cuh"
#include "experts_gemm.h"

namespace skinny {
namespace {

constexpr int kDotWarps = 8;

template <int V, bool SWIGLU>
__global__ void __launch_bounds__(32 * kDotWarps)
experts_dot_kernel(const uint16_t *__restrict__ X, int64_t ldx, int rows, const int32_t *__restrict__ offsets,
                   const uint16_t *__restrict__ W, int64_t ldw, int64_t ldwe, int N, int K, int out_bf16,
                   void *__restrict__ Y, int64_t ldy)
{
    constexpr int NR = SWIGLU ? 2 : 4;        // outputs per warp and row of X
    constexpr int TT = 8;
    griddep_launch_dependents();
    griddep_wait();
    const int e = blockIdx.y;
    const int r0 = max(0, min(rows, __ldcg(offsets + e))), r1 = min(rows, __ldcg(offsets + e + 1));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n0 = (blockIdx.x * kDotWarps + warp) * NR;
    if (n0 >= N) return;
    const uint16_t *w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = min(n0 + i % NR, N - 1);
        w[i] = W + (int64_t)e * ldwe + (int64_t)(SWIGLU && i >= NR ? N + n : n) * ldw;
    }
    for (int r = r0; r < r1; r += TT) {
        float acc[4][TT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < TT; ++m) acc[i][m] = 0.f;
        for (int k0 = 0; k0 < K; k0 += 256) {
            float a[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) load8<V, true>(w[i], k0, K, lane, a[i]);
#pragma unroll
            for (int m = 0; m < TT; ++m) {
                if (r + m >= r1) break;
                float x[8];
                load8<V, false>(X + (int64_t)(r + m) * ldx, k0, K, lane, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) p = fmaf(a[i][j], x[j], p);
                    acc[i][m] += p;
                }
            }
        }
#pragma unroll
        for (int m = 0; m < TT; ++m) {
            if (r + m >= r1) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][m] = warp_sum(acc[i][m]);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float g = acc[i][m];
                const float y = SWIGLU ? g / (1.f + expf(-g)) * acc[(NR + i) & 3][m] : g;
                if (lane == i && n0 + i < N) store_y(Y, out_bf16, (int64_t)(r + m) * ldy + n0 + i, y);
            }
        }
    }
}

template <int V>
cudaError_t launch_dot(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream) {
    const uint16_t *X = a.X, *W = a.W;
    int64_t ldx = a.ldx, ldw = a.ldw, ldwe = a.ldwe, ldy = a.ldy;
    int rows = a.rows, N = a.N, K = a.K, ob = a.out_bf16;
    const int32_t *off = a.offsets;
    void *Y = a.Y;
    void *args[] = {&X, &ldx, &rows, &off, &W, &ldw, &ldwe, &N, &K, &ob, &Y, &ldy};
    const int per = kDotWarps * (a.swiglu ? 2 : 4);
    const void *fn = a.swiglu ? (const void *)experts_dot_kernel<V, true> : (const void *)experts_dot_kernel<V, false>;
    return launch_plain(fn, dim3((N + per - 1) / per, a.E), 32 * kDotWarps, 0, stream, c.pdl, args);
}

}  // namespace

cudaError_t launch_experts_dot(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.W) | (uintptr_t)(2 * a.ldx) |
                          (uintptr_t)(2 * a.ldw) | (uintptr_t)(2 * a.ldwe);
    switch (bf16_vec(all)) {
        case 8: return launch_dot<8>(a, c, stream);
        case 4: return launch_dot<4>(a, c, stream);
        case 2: return launch_dot<2>(a, c, stream);
        default: return launch_dot<1>(a, c, stream);
    }
}

}  // namespace skinny
