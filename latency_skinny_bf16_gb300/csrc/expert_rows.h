// expert_rows.h -- host-side declarations of expert_rows.cu.
#pragma once

#include "calls.h"
#include "skinny_experts.h"

namespace skinny {

constexpr int kMaxTopk = SKINNY_MAX_TOPK;
constexpr int kMaxSortExperts = SKINNY_MAX_SORT_EXPERTS;
constexpr int kSortSmem = 200 * 1024;   // counts of the sort's warps per CTA

struct DispatchArgs {
    const int32_t *ids;
    int64_t ldid;
    const void *X;       // NULL: sort only
    int64_t ldx;
    int T, k, E, H, el_bytes;
    int32_t *pos, *order, *offsets;   // order may be NULL
    void *Xs;
    int64_t ldxs;
};
struct CombineArgs {
    const void *Ys;
    int64_t ldys;
    int rows;
    const int32_t *pos;
    const float *weights;             // NULL: ones
    int64_t ldw;
    int T, k, H;
    bool in16, out16;
    void *Y;
    int64_t ldy;
};
struct CombineGradArgs {
    const void *dY;
    int64_t lddy;
    const void *Ys;
    int64_t ldys;
    int rows;
    const int32_t *pos;
    const float *weights;             // NULL: ones
    int64_t ldw;
    int T, k, H;
    bool b16;
    void *dYs;
    int64_t lddys;
    float *dweights;                  // NULL: not computed
    int64_t lddw;
};

cudaError_t expert_rows_prepare();
cudaError_t launch_dispatch(const DispatchArgs &a, const CallCtx &c, cudaStream_t stream);
cudaError_t launch_combine(const CombineArgs &a, const CallCtx &c, cudaStream_t stream);
cudaError_t launch_combine_grad(const CombineGradArgs &a, const CallCtx &c, cudaStream_t stream);

}  // namespace skinny
