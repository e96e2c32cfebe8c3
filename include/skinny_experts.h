/*
 * skinny_experts.h -- C ABI of what stands around the router and the decode
 * projections in a mixture-of-experts layer: tokens sorted by expert and back
 * with their gradients, the experts' products, and a shared projection with a
 * low-rank adapter per token.  Same conventions as skinny_gemm.h: bf16 as
 * 16-bit patterns, streams as `void*`, every call asynchronous on `stream`,
 * no allocation, no synchronisation (graph-capturable), every argument error
 * found on the host before anything is launched, results bit-identical from
 * run to run on buffers that lie alike within 16 bytes (the dot products of
 * skinny_expert_combine_grad are added in the order of the pieces it stores).
 * Waits inside the kernels are bounded: one that gives up reports
 * SKINNY_ERR_DEVICE_TIMEOUT to skinny_get_device_status.  What its call was to
 * write is then not a result: parts may be written, parts be left as they
 * were, and skinny_lora_gemm_bf16 adds the adapters to what its projection has
 * left.  Nothing else is written, and later calls are not affected.
 *
 * The framework's router gives ids[t][j] (skinny_router_topk).  An entry
 * f = t * k + j is live when 0 <= ids[t][j] < E; any other id (-1, say) drops
 * it: a dropped entry has no row, adds nothing and gets a zero gradient.  A
 * token may have no live entry left.
 */
#ifndef SKINNY_EXPERTS_H_
#define SKINNY_EXPERTS_H_

#include "skinny_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SKINNY_BF16 = 0,
    SKINNY_F32 = 1
} skinny_dtype_t;

typedef enum {
    SKINNY_ACT_NONE = 0,
    SKINNY_ACT_SWIGLU = 1
} skinny_act_t;

#define SKINNY_MAX_TOPK 64            /* entries per token */
#define SKINNY_MAX_SORT_EXPERTS 8192  /* experts of skinny_expert_dispatch */
#define SKINNY_MAX_EXPERTS 1024       /* experts of skinny_experts_gemm_bf16 */
#define SKINNY_MAX_RANK 256           /* columns of an adapter */
#define SKINNY_MAX_WIDTH (1 << 20)    /* elements of a row of X, Ys or dY */

/*
 * Tokens sorted by expert (a stable counting sort of the live entries):
 *
 *     offsets[e]       = number of live entries whose id is below e, e = 0..E
 *     pos[t*k + j]     = offsets[id] + number of live entries f' < t*k + j of the same id; -1 when dropped
 *     order[pos[f]]    = f;  order[p] = -1 for offsets[E] <= p < T*k
 *     Xs[pos[t*k+j],:] = X[t,:]
 *
 *   ids      device, int32 [T, k], row stride ldid >= k
 *   X        device, `dtype` [T, H], row stride ldx >= H, or NULL: sort only (Xs, H, ldx, ldxs, dtype unused)
 *   pos      device, int32 [T*k] written;  order device, int32 [T*k] written, or NULL;
 *   offsets  device, int32 [E + 1] written
 *   Xs       device, `dtype` [T*k, H], row stride ldxs >= H: rows below offsets[E] are written,
 *            the others are left as they are
 *   T >= 0 (0: only offsets are written, all zero), 0 <= k <= 64 (0 as T = 0), 1 <= E <= 8192,
 *   0 <= H <= 2^20, T * k < 2^31.  Outputs overlap neither the inputs nor each other.
 *
 * Errors: INVALID_VALUE (sizes, strides, NULL, dtype, overlap), UNSUPPORTED (k, E, H or T * k too
 * large), MISALIGNED (a pointer not aligned to its element), NO_DEVICE, LAUNCH.
 */
SKINNY_API skinny_status_t skinny_expert_dispatch(const int32_t *ids, int ldid, const void *X, int ldx, int T, int k,
                                                  int E, int H, int dtype, int32_t *pos, int32_t *order,
                                                  int32_t *offsets, void *Xs, int ldxs, void *stream);

/*
 * The experts' rows back to their tokens:
 *
 *     Y[t,:] = sum over j with 0 <= pos[t*k+j] < rows, in order of j, of  weights[t*ldw + j] * Ys[pos[t*k+j],:]
 *
 * summed in fp32 and rounded once to out_dtype; weights == NULL takes 1 (the
 * gradient of skinny_expert_dispatch's copies: dX from dXs).  A token without
 * such an entry gets zeros; the weight of a dropped entry is not used (it may
 * be NaN).
 *
 *   Ys  device, in_dtype [rows, H], row stride ldys >= H;  Y device, out_dtype [T, H], row stride ldy >= H
 *   pos device, int32 [T*k];  weights device, fp32 [T, k], row stride ldw >= k
 *   in_dtype / out_dtype: bf16 -> bf16, fp32 -> fp32, fp32 -> bf16 or bf16 -> fp32.  0 <= k <= 64.
 *   T >= 0, 0 <= H <= 2^20 (0: no-op).  Y overlaps none of the inputs.
 */
SKINNY_API skinny_status_t skinny_expert_combine(const void *Ys, int ldys, int rows, const int32_t *pos,
                                                 const float *weights, int ldw, int T, int k, int H, int in_dtype,
                                                 int out_dtype, void *Y, int ldy, void *stream);

/*
 * The gradient of skinny_expert_combine for dY [T, H]:
 *
 *     dYs[p,:]          = weights[t*ldw + j] * dY[t,:]     for p = pos[t*k+j], 0 <= p < rows
 *     dweights[t*lddw+j] = sum_h dY[t,h] * Ys[p,h]          (fp32; 0 for a dropped entry)
 *
 * dY, Ys and dYs share `dtype`; products and sums in fp32, dYs rounded once.
 * weights == NULL takes 1.  dweights == NULL: not computed, Ys is not read
 * (and may be NULL).  Rows of dYs that no entry names are left as they are.
 */
SKINNY_API skinny_status_t skinny_expert_combine_grad(const void *dY, int lddy, const void *Ys, int ldys, int rows,
                                                      const int32_t *pos, const float *weights, int ldw, int T, int k,
                                                      int H, int dtype, void *dYs, int lddys, float *dweights,
                                                      int lddw, void *stream);

/*
 * The experts' products on rows in expert order: for every expert e and row r
 * with offsets[e] <= r < offsets[e+1],
 *
 *     SKINNY_ACT_NONE:    Y[r,n] = sum_k Xs[r,k] * W[e][n][k]                         n < N, W [E, N, K]
 *     SKINNY_ACT_SWIGLU:  Y[r,n] = g / (1 + exp(-g)) * u,  g = sum_k Xs[r,k] * W[e][n][k],
 *                         u = sum_k Xs[r,k] * W[e][N+n][k]                             n < N, W [E, 2N, K]
 *
 * fp32 accumulation (sums as in skinny_gemm_bf16: bounded tensor-core chains,
 * rounded adds), one rounding to out_dtype.  An expert without rows is not
 * read.  Rows from offsets[E] on are left as they are.
 *
 *   Xs       device, bf16 [rows, K], row stride ldx >= K
 *   offsets  device, int32 [E + 1], non-decreasing, from skinny_expert_dispatch (entries are
 *            clamped to [0, rows])
 *   W        device, bf16, row stride ldw >= K, expert stride ldwe >= (rows of an expert) * ldw (elements)
 *   Y        device, out_dtype [rows, N], row stride ldy >= N; overlaps no input
 *   1 <= E <= 1024; rows, N, K >= 0 (rows or N 0: no-op; K 0: zeros).
 *
 * With 16-byte aligned rows (pointers, ldx, ldw and ldwe multiples of 8
 * elements), more than two rows an expert and enough of N and K the tcgen05
 * kernel runs, else an mma.sync kernel that takes any alignment.  Both take any
 * number of rows for an expert; they are built for decode (up to 64).
 * SKINNY_OPT_FORCE_BACKEND: SKINNY_BACKEND_TCGEN05 is the first (UNSUPPORTED
 * where rows are not aligned), SKINNY_BACKEND_DOTPROD the second.
 */
SKINNY_API skinny_status_t skinny_experts_gemm_bf16(const uint16_t *Xs, int ldx, int rows, const int32_t *offsets,
                                                    const uint16_t *W, int ldw, int64_t ldwe, int E, int N, int K,
                                                    int act, int out_dtype, void *Y, int ldy, void *stream);

/*
 * A shared projection with a low-rank adapter per token beside it: with
 * a = adapters[m] and r_a = ranks[a] (R when ranks == NULL),
 *
 *     Y[m,n] = sum_k X[m,k] W[n,k] + scales[a] * sum_{r < r_a} ( sum_k X[m,k] A[a][r][k] ) * B[a][n][r]
 *
 * A token whose id is outside [0, L) has no adapter.  The inner sum is kept
 * in fp32; Y is rounded once to out_dtype.  What A and B hold past r_a is not
 * used.  ranks are clamped to [0, R]; scales == NULL takes 1.
 *
 *   X, W     as in skinny_gemm_bf16, M <= 64; 16-byte aligned rows (pointers, ldx and ldw multiples of 8
 *            elements) give its results, and rows of any other alignment are taken for every M
 *   A        device, bf16 [L, R, K], row stride lda >= K, adapter stride ldae
 *   B        device, bf16 [L, N, R], row stride ldb >= R, adapter stride ldbe
 *   adapters device, int32 [M];  ranks device, int32 [L] or NULL;  scales device, fp32 [L] or NULL
 *   workspace  device, 16-byte aligned, skinny_lora_workspace(M, N, R, out_dtype) bytes, not shared
 *            with a call that may run at the same time
 *   0 <= R <= 256, L >= 0 (either 0: the projection alone).
 */
SKINNY_API skinny_status_t skinny_lora_gemm_bf16(const uint16_t *X, int ldx, const uint16_t *W, int ldw,
                                                 const uint16_t *A, int lda, int64_t ldae, const uint16_t *B, int ldb,
                                                 int64_t ldbe, const int32_t *adapters, const int32_t *ranks,
                                                 const float *scales, int L, int R, void *Y, int ldy, int M, int N,
                                                 int K, int out_dtype, void *workspace, int64_t workspace_bytes,
                                                 void *stream);

/* Bytes of workspace skinny_lora_gemm_bf16 needs; 0 for sizes it refuses.  Host only. */
SKINNY_API int64_t skinny_lora_workspace(int M, int N, int R, int out_dtype);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_EXPERTS_H_ */
