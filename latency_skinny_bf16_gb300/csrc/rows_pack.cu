// rows_pack.cu -- rows of any alignment laid out on 16-byte boundaries, for the
// tensor maps of the products behind: a copy, whole 16-byte pieces on both sides.
// A warp takes runs of 128 pieces of a row; a lane loads four aligned pieces of
// the source at once and puts each destination piece together from its own and
// the next lane's.  GB300: 4095 x 7167 19 us (6.0 TB/s of reads and writes).
#include "experts_gemm.h"
#include "layer.h"
#include "mma_rows.cuh"

namespace skinny {
namespace {

constexpr int kThreads = 256;

constexpr int kRun = 4;              // pieces of a lane at a time

struct PackParams {
    PackArgs m[2];
    Extent ext[2];
    int runs[2];             // of a row
    int64_t units[2];        // runs of the matrix
};

// The aligned 16 bytes at `at`, as far as they lie inside the extent.
__device__ __forceinline__ uint4 inside16(uintptr_t at, const Extent &ext) {
    if (at >= ext.lo && at + 16 <= ext.hi) return ldg_v4(reinterpret_cast<const void *>(at));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uintptr_t p = at + 2 * e;
        if (p >= ext.lo && p + 2 <= ext.hi) w[e >> 1] |= (uint32_t)ldg_u16(reinterpret_cast<const void *>(p)) << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 from_lane(const uint4 &v, int lane) {
    return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, lane), __shfl_sync(0xFFFFFFFFu, v.y, lane),
                      __shfl_sync(0xFFFFFFFFu, v.z, lane), __shfl_sync(0xFFFFFFFFu, v.w, lane));
}

__global__ void __launch_bounds__(kThreads) rows_pack_kernel(const __grid_constant__ PackParams p)
{
    follow();
    const int lane = threadIdx.x & 31;
    const int64_t all = p.units[0] + p.units[1], warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < all; u += warps) {
        const int w = u >= p.units[0];
        const PackArgs &m = p.m[w];
        const int64_t in = u - (w ? p.units[0] : 0);
        const int64_t r = in / p.runs[w];
        const int per = (m.cols + 7) / 8, c0 = (int)(in - r * p.runs[w]) * 32 * kRun;
        const uintptr_t row = reinterpret_cast<uintptr_t>(m.from + r * m.ldfrom), base = row & ~(uintptr_t)15;
        const int off = (int)(row - base);
        // a piece past the row's last is needed where the row starts off a boundary
        const int need = per + (off != 0);
        uint4 v[kRun + 1];
#pragma unroll
        for (int i = 0; i <= kRun; ++i) {
            const int c = c0 + 32 * i + lane;
            v[i] = make_uint4(0, 0, 0, 0);
            if (c < need && (i < kRun || lane == 0)) v[i] = inside16(base + 16 * (uintptr_t)c, p.ext[w]);
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int c = c0 + 32 * i + lane;
            const uint4 same = from_lane(v[i], lane < 31 ? lane + 1 : 31), first = from_lane(v[i + 1], 0);
            const uint4 next = lane < 31 ? same : first;
            if (c < per) *reinterpret_cast<uint4 *>(m.to + (r * per + c) * 8) = shifted16(v[i], next, off);
        }
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
        p.runs[i] = ((m.cols + 7) / 8 + 32 * kRun - 1) / (32 * kRun);
        p.units[i] = m.rows * p.runs[i];
    }
    const int64_t all = p.units[0] + p.units[1], most = 6ll * c.num_sms, need = (all + kThreads / 32 - 1) / (kThreads / 32);
    if (need == 0) return cudaSuccess;
    void *args[] = {&p};
    return launch_plain((const void *)rows_pack_kernel, dim3((unsigned)(need < most ? need : most)), kThreads, 0, stream, c.pdl, args);
}

}  // namespace skinny
