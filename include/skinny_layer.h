/*
 * skinny_layer.h -- C ABI of a dense layer's operators around the decode
 * projections: a product with bias, activation and residual in its epilogue
 * (both projections of a gated feed-forward block among them), norms of
 * queries and keys for each head with the position rotation in the same pass,
 * and the backward passes of both.  Same conventions as skinny_gemm.h: bf16 as
 * 16-bit patterns, streams as `void*`, every call asynchronous on `stream`, no
 * allocation, no synchronisation (graph-capturable), every argument error found
 * on the host before anything is launched, results bit-identical from run to
 * run on buffers that lie alike within 16 bytes.  Waits inside the kernels are
 * bounded: one that gives up reports SKINNY_ERR_DEVICE_TIMEOUT to
 * skinny_get_device_status, and what its call was to write is then not a result.
 */
#ifndef SKINNY_LAYER_H_
#define SKINNY_LAYER_H_

#include "skinny_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations beside SKINNY_ACT_NONE and SKINNY_ACT_SWIGLU, with
 *   silu(z) = z / (1 + exp(-z)),
 *   gelu(z) = z / (1 + exp(-2 c (z + 0.044715 z^3))),  c = sqrt(2 / pi)   (the tanh form) */
typedef enum {
    SKINNY_ACT_SILU = 2,
    SKINNY_ACT_GELU = 3,
    SKINNY_ACT_GEGLU = 4
} skinny_linear_act_t;

#define SKINNY_MAX_HEAD 512    /* elements of a head */
#define SKINNY_MAX_AXES 8      /* axes of a position */

/*
 * A product with its epilogue.  With Z[m,j] = sum_k X[m,k] W[j,k] + bias[j],
 *
 *     SKINNY_ACT_NONE, SILU, GELU:   Y[m,n] = act(Z[m,n]) + R[m,n]                    W [N, K], bias [N]
 *     SKINNY_ACT_SWIGLU, GEGLU:      Y[m,n] = act(Z[m,n]) * Z[m,N+n] + R[m,n]         W [2N, K], bias [2N]
 *                                    (act is silu or gelu: gates, then ups)
 *
 * Sums in fp32 (tensor-core chains of at most 16 MMAs, or 64 where there are
 * many rows, then rounded adds): within 1e-5 of sum_k |x w| up to a depth of
 * 32768, as in skinny_gemm_bf16, and by 2^-32 of it more for each step of the
 * depth beyond (2.5e-4 at the deepest, K = 2^20).  The epilogue in fp32, one
 * rounding to out_dtype.  Z, for the backward pass, is rounded to bf16 beside
 * it; Y is computed from what was not rounded.
 *
 *   X     device, bf16 [M, K], row stride ldx >= K;  W  device, bf16, row stride ldw >= K
 *   bias  device, bf16 [N or 2N], or NULL;  R  device, out_dtype [M, N], row stride ldr >= N, or NULL
 *   Y     device, out_dtype [M, N], row stride ldy >= N.  R may be Y itself (same row stride);
 *         otherwise Y and Z overlap no input and not each other.  Columns of one buffer side by side (one
 *         row stride) do not overlap.
 *   Z     device, bf16 [M, N or 2N], row stride ldz, or NULL
 *   workspace  device, 16-byte aligned, skinny_linear_workspace(...) bytes for the same arguments, not
 *         shared with a call that may run at the same time; NULL where that is 0
 *   M >= 0; 0 <= N, K <= 2^20.  M or N 0: no-op.  K 0: the empty sum.
 *
 * Rows that are not 16-byte aligned (pointer, ldx, ldw multiples of 8 elements) are taken too: they are
 * laid out in the workspace first, which is 0 bytes without such rows.
 *
 * Unlike skinny_gemm_bf16, W may be written by the kernel just before on the stream, with PDL on as well.
 *
 * SKINNY_OPT_FORCE_BACKEND, also for the products of the backward pass: SKINNY_BACKEND_TCGEN05 is the
 * kernel by pairs of SMs, SKINNY_BACKEND_SPLITK the one with the depth split over a cluster.
 *
 * Errors: INVALID_VALUE (sizes, strides, NULL, act, dtype, overlap, workspace too small), UNSUPPORTED
 * (N or K too large), MISALIGNED (a pointer not aligned to its element, the workspace), NO_DEVICE, LAUNCH.
 */
SKINNY_API skinny_status_t skinny_linear_bf16(const uint16_t *X, int ldx, const uint16_t *W, int ldw,
                                              const uint16_t *bias, const void *R, int ldr, void *Y, int ldy,
                                              uint16_t *Z, int ldz, int M, int N, int K, int act, int out_dtype,
                                              void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace skinny_linear_bf16 needs for these arguments; 0 for sizes it refuses.  Host only. */
SKINNY_API int64_t skinny_linear_workspace(const uint16_t *X, int ldx, const uint16_t *W, int ldw, int M, int N,
                                           int K, int act);

/*
 * The gradients of skinny_linear_bf16 for dY [M, N], from the Z that it kept:
 *
 *     dZ[m,n] = dY[m,n] act'(Z[m,n]);  gated:  dZ[m,n] = dY[m,n] Z[m,N+n] act'(Z[m,n]),  dZ[m,N+n] = dY[m,n] act(Z[m,n])
 *     dX[m,k] = sum_j dZ[m,j] W[j,k],   dW[j,k] = sum_m dZ[m,j] X[m,k],   dbias[j] = sum_m dZ[m,j]
 *
 * (R's gradient is dY.)  dZ is computed in fp32 and rounded to bf16 for the two
 * products, as the tensor cores take it; dbias sums what was not rounded.  Sums
 * in fp32 as above, over a depth of N or 2N (dX) or M tokens (dW, dbias), one
 * rounding of dX and dW to bf16.  SKINNY_ACT_NONE needs no Z (NULL), and dZ is
 * dY itself.
 *
 *   dY  device, bf16 [M, N];  X, W as above;  Z  device, bf16 [M, N or 2N]
 *   dX  device, bf16 [M, K], or NULL: not computed (W may then be NULL)
 *   dW  device, bf16 [N or 2N, K], or NULL: not computed (X may then be NULL)
 *   dbias  device, fp32 [N or 2N], or NULL
 *   Outputs overlap neither the inputs nor each other.
 *   M 0: dW and dbias are zeros.  N 0: dX is zeros.
 */
SKINNY_API skinny_status_t skinny_linear_grad_bf16(const uint16_t *dY, int lddy, const uint16_t *X, int ldx,
                                                   const uint16_t *W, int ldw, const uint16_t *Z, int ldz,
                                                   uint16_t *dX, int lddx, uint16_t *dW, int lddw, float *dbias,
                                                   int M, int N, int K, int act, void *workspace,
                                                   int64_t workspace_bytes, void *stream);

/* Bytes of workspace skinny_linear_grad_bf16 needs for these arguments (whichever gradients are asked
 * for); 0 for sizes it refuses.  Host only. */
SKINNY_API int64_t skinny_linear_grad_workspace(const uint16_t *dY, int lddy, const uint16_t *X, int ldx,
                                                const uint16_t *W, int ldw, int M, int N, int K, int act);

/* Heads of queries or keys: `dtype` [T, H, D], token stride st and head stride sh in elements, unit
 * stride along D.  Heads do not overlap: sh >= D and st >= (H - 1) sh + D, or the other way round. */
typedef struct {
    const void *x;
    int64_t st, sh;
    const void *w;       /* the norm's weight, `dtype` [D], or NULL: ones */
    int H;
} skinny_heads_t;

/* How heads are turned: pair i < R / 2 of a head holds elements (i, R/2 + i), or (2i, 2i + 1) when
 * interleaved; the elements from R on are not turned. */
typedef struct {
    const float *table;        /* device, fp32 [P, R], row stride R: cos of the R / 2 pairs, then sin */
    int64_t P;                 /* positions of the table */
    const int32_t *positions;  /* device, int32 [axes, T] */
    const int32_t *pair_axis;  /* device, int32 [R / 2]: the axis that turns each pair; NULL: axis 0 */
    int axes, R, interleaved;
} skinny_rotation_t;

/*
 * Norms of queries and keys for each head, and the position rotation, in one pass:
 *
 *     n[d] = x[d] / sqrt(sum_d x[d]^2 / D + eps) * w[d]         (norm != 0; else n = x)
 *     y[a] = n[a] c - n[b] s,  y[b] = n[b] c + n[a] s           for each pair (a, b), c and s the table's
 *                                                               entries at the token's position on the pair's axis
 *
 * in fp32, rounded once to dtype.  A position outside [0, P), or an axis outside [0, axes), does not
 * turn its pairs (padding may hold -1).  NaN and infinite elements stay within their head.
 *
 *   q, k     the inputs; H 0: none of the kind (its pointers are not used)
 *   q_out    device, dtype [T, q.H, D], strides q_st, q_sh; k_out likewise.  An output may be its own input
 *            (same pointer and strides); otherwise it overlaps no input and not the other output.  Views that
 *            share a token stride may lie beside each other in each token, and heads may take turns, a query's
 *            beside its key's, where all strides are multiples of the smallest.
 *   T >= 0, 1 <= D <= 512, 0 <= R <= D even (0: no rotation, the table is not used), 1 <= axes <= 8, 1 <= P.
 */
SKINNY_API skinny_status_t skinny_qk_norm_rope(const skinny_heads_t *q, const skinny_heads_t *k,
                                               const skinny_rotation_t *rot, int T, int D, int norm, float eps,
                                               int dtype, void *q_out, int64_t q_st, int64_t q_sh, void *k_out,
                                               int64_t k_st, int64_t k_sh, void *stream);

/*
 * Its gradients for dq [T, q.H, D] and dk: with g the rows of dq turned back, h = g w and
 * r = 1 / sqrt(sum_d x[d]^2 / D + eps),
 *
 *     dx[d] = r h[d] - x[d] r^3 sum_d(h[d] x[d]) / D            (norm == 0: dx = g, x is not read)
 *     dw[d] = sum over tokens and heads of g[d] x[d] r          (fp32, in a fixed order)
 *
 *   dq, dk       inputs, dtype, strides dq_st, dq_sh and dk_st, dk_sh
 *   q_grad       device, dtype [T, q.H, D], strides qg_st, qg_sh (it may be dq itself); k_grad likewise
 *   q_wgrad, k_wgrad  device, fp32 [D] written, or NULL: not computed (norm == 0: they are NULL)
 *   workspace    device, 16-byte aligned, skinny_qk_norm_rope_grad_workspace(T, q.H, k.H, D) bytes, not shared
 *                with a call that may run at the same time; not used without weight gradients
 */
SKINNY_API skinny_status_t skinny_qk_norm_rope_grad(const void *dq, int64_t dq_st, int64_t dq_sh, const void *dk,
                                                    int64_t dk_st, int64_t dk_sh, const skinny_heads_t *q,
                                                    const skinny_heads_t *k, const skinny_rotation_t *rot, int T,
                                                    int D, int norm, float eps, int dtype, void *q_grad,
                                                    int64_t qg_st, int64_t qg_sh, void *k_grad, int64_t kg_st,
                                                    int64_t kg_sh, float *q_wgrad, float *k_wgrad, void *workspace,
                                                    int64_t workspace_bytes, void *stream);

/* Bytes of workspace of skinny_qk_norm_rope_grad; 0 for sizes it refuses.  Host only. */
SKINNY_API int64_t skinny_qk_norm_rope_grad_workspace(int T, int q_heads, int k_heads, int D);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_LAYER_H_ */
