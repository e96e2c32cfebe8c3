// experts_api.cu -- the C ABI of skinny_experts.h: argument checks and
// launches.  Every argument is checked on the host before anything is
// launched; no entry point throws, allocates or synchronises.
#include <initializer_list>

#include "calls.h"
#include "expert_rows.h"
#include "experts_gemm.h"
#include "skinny_experts.h"

namespace skinny {
namespace {

int el_bytes(int dtype) { return dtype == SKINNY_BF16 ? 2 : 4; }
bool dtype_ok(int d) { return d == SKINNY_BF16 || d == SKINNY_F32; }
uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
bool aligned(const void *p, int bytes) { return addr(p) % (uintptr_t)bytes == 0; }

// The bytes [lo, hi) that a matrix of `rows` rows of `cols` elements occupies.
struct Range {
    uintptr_t lo, hi;
};
Range span(const void *p, int64_t rows, int64_t cols, int64_t ld, int el) {
    if (!p || rows <= 0 || cols <= 0) return {0, 0};
    return {addr(p), addr(p) + (uintptr_t)(((rows - 1) * ld + cols) * el)};
}
// Whether a range that is written meets one of the others.
bool meets(const Range &w, std::initializer_list<Range> others) {
    for (const Range &o : others)
        if (w.lo < w.hi && o.lo < o.hi && ranges_overlap(w.lo, w.hi, o.lo, o.hi)) return true;
    return false;
}

skinny_status_t launched(cudaError_t e) { return e == cudaSuccess ? SKINNY_OK : SKINNY_ERR_LAUNCH; }

// T, k and H of a call on the router's entries.
skinny_status_t check_entries(int T, int k, int H) {
    if (T < 0 || k < 0 || H < 0) return SKINNY_ERR_INVALID_VALUE;
    if (k > kMaxTopk || (int64_t)T * k >= (1ll << 31) || H > SKINNY_MAX_WIDTH) return SKINNY_ERR_UNSUPPORTED;
    return SKINNY_OK;
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

skinny_status_t skinny_expert_dispatch(const int32_t *ids, int ldid, const void *X, int ldx, int T, int k, int E,
                                       int H, int dtype, int32_t *pos, int32_t *order, int32_t *offsets, void *Xs,
                                       int ldxs, void *stream) {
    skinny_status_t st = check_entries(T, k, X ? H : 0);
    if (st != SKINNY_OK) return st;
    if (E < 1) return SKINNY_ERR_INVALID_VALUE;
    if (E > kMaxSortExperts) return SKINNY_ERR_UNSUPPORTED;
    if (!offsets) return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(offsets, 4)) return SKINNY_ERR_MISALIGNED;
    if (k == 0) T = 0;
    DispatchArgs a{ids, ldid, nullptr, 0, T, k, E, 0, 2, pos, order, offsets, nullptr, 0};
    if (T > 0) {
        const int64_t n = (int64_t)T * k;
        if (!ids || !pos || ldid < k) return SKINNY_ERR_INVALID_VALUE;
        if (!aligned(ids, 4) || !aligned(pos, 4) || !aligned(order, 4)) return SKINNY_ERR_MISALIGNED;
        Range x{0, 0}, xs{0, 0};
        if (X && H != 0) {
            if (!dtype_ok(dtype) || !Xs || ldx < H || ldxs < H) return SKINNY_ERR_INVALID_VALUE;
            const int b = el_bytes(dtype);
            if (!aligned(X, b) || !aligned(Xs, b)) return SKINNY_ERR_MISALIGNED;
            x = span(X, T, H, ldx, b);
            xs = span(Xs, n, H, ldxs, b);
            a.X = X; a.ldx = ldx; a.H = H; a.el_bytes = b; a.Xs = Xs; a.ldxs = ldxs;
        }
        const Range i = span(ids, T, k, ldid, 4), p = span(pos, 1, n, n, 4), o = span(order, 1, n, n, 4),
                    f = span(offsets, 1, E + 1, E + 1, 4);
        if (meets(xs, {x, i, p, o, f}) || meets(p, {x, i, o, f}) || meets(o, {x, i, f}) || meets(f, {x, i}))
            return SKINNY_ERR_INVALID_VALUE;
    }
    CallCtx c;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    return launched(launch_dispatch(a, c, static_cast<cudaStream_t>(stream)));
}

skinny_status_t skinny_expert_combine(const void *Ys, int ldys, int rows, const int32_t *pos, const float *weights,
                                      int ldw, int T, int k, int H, int in_dtype, int out_dtype, void *Y, int ldy,
                                      void *stream) {
    skinny_status_t st = check_entries(T, k, H);
    if (st != SKINNY_OK) return st;
    if (rows < 0 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return SKINNY_ERR_INVALID_VALUE;
    if (T == 0 || H == 0) return SKINNY_OK;
    const int ib = el_bytes(in_dtype), ob = el_bytes(out_dtype);
    if (!Y || ldy < H) return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(Y, ob)) return SKINNY_ERR_MISALIGNED;
    if (k > 0) {
        if (!pos || (rows > 0 && (!Ys || ldys < H)) || (weights && ldw < k)) return SKINNY_ERR_INVALID_VALUE;
        if (!aligned(pos, 4) || !aligned(weights, 4) || !aligned(Ys, ib)) return SKINNY_ERR_MISALIGNED;
        if (meets(span(Y, T, H, ldy, ob), {span(Ys, rows, H, ldys, ib), span(pos, 1, (int64_t)T * k, 0, 4),
                                           span(weights, T, k, ldw, 4)}))
            return SKINNY_ERR_INVALID_VALUE;
    }
    CallCtx c;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    const CombineArgs a{Ys, ldys, rows, pos, weights, ldw, T, k, H, in_dtype == SKINNY_BF16, out_dtype == SKINNY_BF16,
                        Y, ldy};
    return launched(launch_combine(a, c, static_cast<cudaStream_t>(stream)));
}

skinny_status_t skinny_expert_combine_grad(const void *dY, int lddy, const void *Ys, int ldys, int rows,
                                           const int32_t *pos, const float *weights, int ldw, int T, int k, int H,
                                           int dtype, void *dYs, int lddys, float *dweights, int lddw, void *stream) {
    skinny_status_t st = check_entries(T, k, H);
    if (st != SKINNY_OK) return st;
    if (rows < 0 || !dtype_ok(dtype)) return SKINNY_ERR_INVALID_VALUE;
    if (T == 0 || k == 0 || (H == 0 && !dweights)) return SKINNY_OK;
    const int b = el_bytes(dtype);
    if (!pos || (weights && ldw < k) || (dweights && lddw < k)) return SKINNY_ERR_INVALID_VALUE;
    if (H > 0 && (!dY || lddy < H || (rows > 0 && (!dYs || lddys < H)) ||
                  (rows > 0 && dweights && (!Ys || ldys < H))))
        return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(pos, 4) || !aligned(weights, 4) || !aligned(dweights, 4) || !aligned(dY, b) || !aligned(dYs, b) ||
        (dweights && !aligned(Ys, b)))
        return SKINNY_ERR_MISALIGNED;
    const Range g = span(dY, T, H, lddy, b), y = dweights ? span(Ys, rows, H, ldys, b) : Range{0, 0},
                p = span(pos, 1, (int64_t)T * k, 0, 4), w = span(weights, T, k, ldw, 4),
                gy = span(dYs, rows, H, lddys, b), gw = span(dweights, T, k, lddw, 4);
    if (meets(gy, {g, y, p, w, gw}) || meets(gw, {g, y, p, w})) return SKINNY_ERR_INVALID_VALUE;
    CallCtx c;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    const CombineGradArgs a{dY, lddy, Ys, ldys, rows, pos, weights, ldw, T, k, H, dtype == SKINNY_BF16, dYs, lddys,
                            dweights, lddw};
    return launched(launch_combine_grad(a, c, static_cast<cudaStream_t>(stream)));
}

skinny_status_t skinny_experts_gemm_bf16(const uint16_t *Xs, int ldx, int rows, const int32_t *offsets,
                                         const uint16_t *W, int ldw, int64_t ldwe, int E, int N, int K, int act,
                                         int out_dtype, void *Y, int ldy, void *stream) {
    if (E < 1 || rows < 0 || N < 0 || K < 0 || !dtype_ok(out_dtype) ||
        (act != SKINNY_ACT_NONE && act != SKINNY_ACT_SWIGLU))
        return SKINNY_ERR_INVALID_VALUE;
    if (E > SKINNY_MAX_EXPERTS || N > SKINNY_MAX_WIDTH || K > SKINNY_MAX_WIDTH) return SKINNY_ERR_UNSUPPORTED;
    if (rows == 0 || N == 0) return SKINNY_OK;
    const int ob = el_bytes(out_dtype);
    const int64_t wrows = act == SKINNY_ACT_SWIGLU ? 2ll * N : N;
    if (E == 1) ldwe = wrows * ldw;     // no other expert: the stride is not used
    if (!offsets || !Y || ldy < N) return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(offsets, 4) || !aligned(Y, ob)) return SKINNY_ERR_MISALIGNED;
    const Range y = span(Y, rows, N, ldy, ob);
    if (meets(y, {span(offsets, 1, E + 1, 0, 4)})) return SKINNY_ERR_INVALID_VALUE;
    if (K > 0) {
        if (!Xs || !W || ldx < K || ldw < K || (E > 1 && ldwe < wrows * ldw)) return SKINNY_ERR_INVALID_VALUE;
        if (!aligned(Xs, 2) || !aligned(W, 2)) return SKINNY_ERR_MISALIGNED;
        // the experts' matrices: E - 1 strides and the last one's rows
        const Range w = {addr(W), addr(W) + (uintptr_t)(2 * ((E - 1) * ldwe + (wrows - 1) * ldw + K))};
        if (meets(y, {span(Xs, rows, K, ldx, 2), w})) return SKINNY_ERR_INVALID_VALUE;
    }
    CallCtx c;
    const skinny_status_t st = call_context(&c);
    if (st != SKINNY_OK) return st;
    const ExpertsArgs a{Xs, ldx, rows, offsets, W, ldw, ldwe, E, N, K, act == SKINNY_ACT_SWIGLU,
                        out_dtype == SKINNY_BF16, Y, ldy};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.force_backend == SKINNY_BACKEND_TCGEN05)
        return experts_tc_supported(a) ? launched(launch_experts_tc(a, c, s)) : SKINNY_ERR_UNSUPPORTED;
    const bool tc = c.force_backend != SKINNY_BACKEND_DOTPROD && experts_tc_supported(a) && experts_tc_faster(a, c.num_sms);
    return launched(tc ? launch_experts_tc(a, c, s) : launch_experts_mma(a, c, s));
}

int64_t skinny_lora_workspace(int M, int N, int R, int out_dtype) {
    if (M < 0 || M > SKINNY_MAX_M || N < 0 || R < 0 || R > SKINNY_MAX_RANK || !dtype_ok(out_dtype)) return 0;
    // V, then (bf16 output) the projection in fp32 that the adapters are added to before the one rounding
    return (int64_t)M * 3 * lora_padded_rank(R) * 2 + (out_dtype == SKINNY_BF16 ? (int64_t)M * N * 4 : 0);
}

skinny_status_t skinny_lora_gemm_bf16(const uint16_t *X, int ldx, const uint16_t *W, int ldw, const uint16_t *A,
                                      int lda, int64_t ldae, const uint16_t *B, int ldb, int64_t ldbe,
                                      const int32_t *adapters, const int32_t *ranks, const float *scales, int L, int R,
                                      void *Y, int ldy, int M, int N, int K, int out_dtype, void *workspace,
                                      int64_t workspace_bytes, void *stream) {
    if (L < 0 || R < 0 || !dtype_ok(out_dtype)) return SKINNY_ERR_INVALID_VALUE;
    if (R > SKINNY_MAX_RANK) return SKINNY_ERR_UNSUPPORTED;
    const int ob = out_dtype == SKINNY_BF16;
    const bool none = L == 0 || R == 0 || M <= 0 || N <= 0 || K <= 0;
    skinny_status_t st = SKINNY_OK;
    // The projection: skinny_gemm_bf16 where its rows are 16-byte aligned; else the experts' mma.sync
    // kernel on the one matrix, which reads whole 16-byte pieces at any alignment and takes every M.  GB300,
    // us, skinny_gemm_bf16 and this kernel: 896 x 2645, 1, 2, 8 and 16 tokens 10.7 and 11.1, 14.0 and 11.6,
    // 58.9 and 11.1, 102 and 15.3; 15936 x 4083, 1 and 8 tokens 107 and 38, 1500 and 40; short and long the
    // other way round for few tokens, 512 x 7169, 1, 2 and 4 tokens 12.0 and 21.9, 17.6 and 22.9, 53 and 23.
    const bool rows16 = ((addr(X) | addr(W)) % 16 | (ldx | ldw) % 8) == 0;
    if (none) {
        st = run_gemm(X, ldx, W, ldw, Y, ldy, M, N, K, stream, ob);
        // what it refuses of checked arguments: unaligned rows with more than 16 tokens
        if (st != SKINNY_ERR_UNSUPPORTED || M > SKINNY_MAX_M || rows16) return st;
        CallCtx c;
        st = call_context(&c);
        if (st != SKINNY_OK) return st;
        const ExpertsArgs b{X, ldx, M, nullptr, W, ldw, (int64_t)N * ldw, 1, N, K, 0, ob, Y, ldy};
        return launched(launch_experts_mma(b, c, static_cast<cudaStream_t>(stream)));
    }
    if (M > SKINNY_MAX_M) return SKINNY_ERR_UNSUPPORTED;
    if (!Y || ldy < N || !A || !B || !adapters || !workspace || lda < K || ldb < R ||
        (L > 1 && (ldae < (int64_t)R * lda || ldbe < (int64_t)N * ldb)) ||
        workspace_bytes < skinny_lora_workspace(M, N, R, out_dtype))
        return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(Y, el_bytes(out_dtype)) || !aligned(A, 2) || !aligned(B, 2) || !aligned(adapters, 4) ||
        !aligned(ranks, 4) || !aligned(scales, 4) || !aligned(workspace, 16))
        return SKINNY_ERR_MISALIGNED;
    uint16_t *V = static_cast<uint16_t *>(workspace);
    float *base = ob ? reinterpret_cast<float *>(V + (int64_t)M * 3 * lora_padded_rank(R)) : static_cast<float *>(Y);
    const int ldbase = ob ? N : ldy;
    const Range y = span(Y, M, N, ldy, el_bytes(out_dtype)), x = span(X, M, K, ldx, 2), w = span(W, N, K, ldw, 2),
                ws = {addr(workspace), addr(workspace) + (uintptr_t)skinny_lora_workspace(M, N, R, out_dtype)},
                ra = {addr(A), addr(A) + (uintptr_t)(2 * ((L - 1) * ldae + (int64_t)(R - 1) * lda + K))},
                rb = {addr(B), addr(B) + (uintptr_t)(2 * ((L - 1) * ldbe + (int64_t)(N - 1) * ldb + R))},
                id = span(adapters, 1, M, 0, 4), rk = span(ranks, 1, L, 0, 4), sc = span(scales, 1, L, 0, 4);
    if (meets(y, {x, w, ws, ra, rb, id, rk, sc}) || meets(ws, {x, w, ra, rb, id, rk, sc}))
        return SKINNY_ERR_INVALID_VALUE;
    if (!X || !W || ldx < K || ldw < K) return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(X, 2) || !aligned(W, 2)) return SKINNY_ERR_MISALIGNED;
    if (rows16) {
        st = check_gemm(X, ldx, W, ldw, base, ldbase, M, N, K, 0);
        if (st != SKINNY_OK) return st;
    }
    CallCtx c;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    const LoraArgs a{X, ldx, A, lda, ldae, B, ldb, ldbe, adapters, ranks, scales, L, R, M, N, K, V, base, ldbase, Y,
                     ldy, ob};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the projection, the shrink beside it, the expand behind both (lora.cu says what may overlap)
    if (rows16) {
        st = run_gemm(X, ldx, W, ldw, base, ldbase, M, N, K, stream, 0, false);
        if (st != SKINNY_OK) return st;
    } else {
        CallCtx plain = c;
        plain.pdl = false;
        const ExpertsArgs b{X, ldx, M, nullptr, W, ldw, (int64_t)N * ldw, 1, N, K, 0, 0, base, ldbase};
        if (launch_experts_mma(b, plain, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
    }
    if (launch_lora_shrink(a, c, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
    return launched(launch_lora_expand(a, c, s));
}

}  // extern "C"
