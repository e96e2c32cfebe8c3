// layer.h -- host-side declarations of a dense layer's operators: products with
// an epilogue and their gradients, heads' norms with rotation and theirs.
#pragma once

#include "calls.h"
#include "skinny_layer.h"

namespace skinny {

// An operand of a product over a depth c: element (i, c) at p[i * ld + c], or,
// crossed, at p[c * ld + i].
struct Operand {
    const uint16_t *p;
    int64_t ld;
    bool crossed;
};

// These kernels let the next of the stream start (programmatic dependent launch) once what precedes themselves is done.
// One that needs nothing of its predecessor in the same call is marked `beside`: it starts at once, as its successor in
// the call does, and waits for the predecessor at its own end, so that what follows may take both as done.  So run, in a
// backward pass, dz beside the laying out of rows, the input's gradient beside the last sums of the bias gradient, the
// weight's beside the input's last tiles.  GB300, us, the two products one behind the other and so: 3000 rows
// 4096 x 2048 74.5 and 63.7, 1500 rows 1500 x 1500 GELU 41.3 and 30.9, 300 rows 600 x 700 17.7 and 13.6; where the tiles
// fill the GPU, the same (2048 x 2048 x 2048 34.3 and 34.3).  The other two, with a bias gradient: 4099 rows 1437 x 2049
// SiLU 98 and 92.7, 33 rows 513 x 511 GELU 13.1 and 11.1.  The last of a call lets the next start at its end only: 64 rows
// SwiGLU 2048 x 7168 47.3, from its start 52.0.
// Y[r][n] = epilogue(sum_c B(r, c) A(n, c)), r < rows, n < cols.  A gated
// activation takes A(cols + n, c) beside it.
struct ProductArgs {
    Operand A, B;
    int64_t rows;
    int cols, depth;
    int act;
    const uint16_t *bias;    // NULL: none
    const void *R;           // out's type; NULL: none
    int64_t ldr;
    void *Y;
    int64_t ldy;
    uint16_t *Z;             // NULL: not kept
    int64_t ldz;
    int out_bf16;
    bool beside;             // of the kernel before: nothing of it is read or written
    bool last;               // of a call; read with beside
};
// 64-step boxes of a depth, which may be the largest int: a gradient's depth is the number of tokens
constexpr int depth_boxes(int depth) { return depth / 64 + (depth % 64 != 0); }
// a depth of 0 (linear_empty.cu)
cudaError_t launch_linear_empty(const ProductArgs &a, const CallCtx &c, cudaStream_t stream);

// tcgen05 (linear_tc.cu): 16-byte aligned rows, a depth of 1 at least
cudaError_t linear_tc_prepare();
int64_t linear_tc_ns(const ProductArgs &a, int num_sms);
cudaError_t launch_linear_tc(const ProductArgs &a, const CallCtx &c, cudaStream_t stream);

// tcgen05 by pairs of SMs (linear_pair.cu), as above
cudaError_t linear_pair_prepare();
bool linear_pair_faster(const ProductArgs &a, int num_sms);   // than linear_tc.cu
cudaError_t launch_linear_pair(const ProductArgs &a, const CallCtx &c, cudaStream_t stream);

// Rows laid out from `to` on, whole 16-byte pieces each; from NULL: none.
struct PackArgs {
    const uint16_t *from;
    int64_t ldfrom, rows;
    int cols;
    uint16_t *to;
};
cudaError_t launch_rows_pack(const PackArgs &a, const PackArgs &b, const CallCtx &c, cudaStream_t stream);

// dZ (bf16, row stride lddz) and, into `partial` [parts][rows of W], the sums of dZ over the tokens of a part
struct LinearDzArgs {
    const uint16_t *dY;
    int64_t lddy;
    const uint16_t *Z;
    int64_t ldz;
    uint16_t *dZ;            // NULL: sums only
    int64_t lddz;
    float *dbias;            // NULL: not computed
    float *partial;          // kDbiasParts rows
    int64_t M;
    int N, act;
    bool beside;
};
constexpr int kDbiasParts = 64;
inline int dbias_parts(int64_t M) {      // four rows a thread of eight at least, what it loads at once
    const int64_t want = (M + 31) / 32;
    return want < kDbiasParts ? (int)want : kDbiasParts;
}
cudaError_t launch_linear_dz(const LinearDzArgs &a, const CallCtx &c, cudaStream_t stream);

// Heads of queries (side 0) and keys (side 1).
struct HeadsSide {
    const void *x;
    int64_t st, sh;
    const void *w;
    const void *d;           // gradients: of the outputs
    int64_t dst, dsh;
    void *y;                 // outputs; gradients: of the inputs
    int64_t yst, ysh;
    float *dw;               // gradients of the weights, or NULL
    int H;
};
struct HeadsArgs {
    HeadsSide side[2];
    const float *table;
    int64_t P;
    const int32_t *positions, *pair_axis;
    int axes, R, interleaved;
    int T, D, norm;
    float eps;
    bool b16, grad;
    float *partial;          // gradients of the weights: [parts][2][D]
};
constexpr int kHeadsParts = 608;
cudaError_t heads_prepare();
cudaError_t launch_heads(const HeadsArgs &a, const CallCtx &c, cudaStream_t stream);

}  // namespace skinny
