// rows_pack.cu -- rows of any alignment laid out on 16-byte boundaries, for the
// tensor maps of the products behind: a copy, whole 16-byte pieces on both sides
// (a piece of the source is put together from the two that hold it).
#include "experts_gemm.h"
#include "layer.h"
#include "mma_rows.cuh"

namespace skinny {
namespace {

constexpr int kThreads = 256;

struct PackParams {
    PackArgs m[2];
    Extent ext[2];
    int64_t pieces[2];       // 16-byte pieces of each destination
};

__global__ void __launch_bounds__(kThreads) rows_pack_kernel(const __grid_constant__ PackParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int64_t all = p.pieces[0] + p.pieces[1];
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads) {
        const int w = i >= p.pieces[0];
        const PackArgs &m = p.m[w];
        const int64_t at = i - (w ? p.pieces[0] : 0);
        const int per = (m.cols + 7) / 8;
        const int64_t r = at / per;
        const int c = (int)(at - r * per) * 8;
        const uint4 v = load_row8<false, false>(m.from + r * m.ldfrom, c, m.cols, p.ext[w]);
        *reinterpret_cast<uint4 *>(m.to + r * per * 8 + c) = v;
    }
}

}  // namespace

cudaError_t launch_rows_pack(const PackArgs &a, const PackArgs &b, const CallCtx &c, cudaStream_t stream) {
    PackParams p{};
    p.m[0] = a;
    p.m[1] = b;
    for (int i = 0; i < 2; ++i) {
        const PackArgs &m = p.m[i];
        if (!m.from) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(m.from);
        p.ext[i] = {lo, lo + (uintptr_t)(2 * ((m.rows - 1) * m.ldfrom + m.cols))};
        p.pieces[i] = m.rows * ((m.cols + 7) / 8);
    }
    const int64_t all = p.pieces[0] + p.pieces[1], most = 8ll * c.num_sms, need = (all + kThreads - 1) / kThreads;
    if (need == 0) return cudaSuccess;
    void *args[] = {&p};
    return launch_plain((const void *)rows_pack_kernel, dim3((unsigned)(need < most ? need : most)), kThreads, 0, stream, c.pdl, args);
}

}  // namespace skinny
