// experts_gemm.h -- host-side declarations of the experts' products and of the
// adapters beside a projection.
#pragma once

#include "calls.h"
#include "skinny_experts.h"

namespace skinny {

struct ExpertsArgs {
    const uint16_t *X;
    int64_t ldx;
    int rows;
    const int32_t *offsets;
    const uint16_t *W;
    int64_t ldw, ldwe;   // row stride, expert stride (elements)
    int E, N, K;
    int swiglu;          // W holds 2N rows an expert: gates, then ups
    int out_bf16;
    void *Y;
    int64_t ldy;
};
// mma.sync, any alignment (experts_mma.cu); K == 0 included
cudaError_t launch_experts_mma(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream);

// tcgen05 (experts_tc.cu): 16-byte aligned rows of X and W, K >= 1
bool experts_tc_supported(const ExpertsArgs &a);
bool experts_tc_faster(const ExpertsArgs &a, int num_sms);   // than the mma.sync kernel
cudaError_t experts_tc_prepare();
cudaError_t launch_experts_tc(const ExpertsArgs &a, const CallCtx &c, cudaStream_t stream);

// Columns of a token's V: whole MMA steps.
__host__ __device__ constexpr int lora_padded_rank(int R) { return (R + 31) / 32 * 32; }
struct LoraArgs {
    const uint16_t *X;
    int64_t ldx;
    const uint16_t *A;
    int64_t lda, ldae;
    const uint16_t *B;
    int64_t ldb, ldbe;
    const int32_t *adapters, *ranks;
    const float *scales;
    int L, R, M, N, K;
    uint16_t *V;         // [M][3][lora_padded_rank(R)], written by the first kernel, read by the second
    const float *base;   // fp32 [M, N] of the shared projection, row stride ldbase
    int64_t ldbase;
    void *Y;             // base itself (fp32), or bf16
    int64_t ldy;
    int out_bf16;
};
cudaError_t launch_lora_shrink(const LoraArgs &a, const CallCtx &c, cudaStream_t stream);
cudaError_t launch_lora_expand(const LoraArgs &a, const CallCtx &c, cudaStream_t stream);

// cluster_z: CTAs of a cluster along the grid's z
inline cudaError_t launch_plain(const void *fn, dim3 grid, int threads, int smem, cudaStream_t stream, bool pdl,
                                void **args, int cluster_z = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = cluster_z;
    cfg.attrs = attr;
    cfg.numAttrs = cluster_z > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace skinny
