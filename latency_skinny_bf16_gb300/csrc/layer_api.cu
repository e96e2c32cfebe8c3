// layer_api.cu -- the C ABI of skinny_layer.h: argument checks and launches.
// Every argument is checked on the host before anything is launched; no entry
// point throws, allocates or synchronises.
#include "act.cuh"
#include "layer.h"
#include "ranges.h"

namespace skinny {
namespace {

bool act_ok(int act) { return act >= SKINNY_ACT_NONE && act <= SKINNY_ACT_GEGLU; }
int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t pad16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

skinny_status_t check_product(int M, int N, int K, int act) {
    if (M < 0 || N < 0 || K < 0 || !act_ok(act)) return SKINNY_ERR_INVALID_VALUE;
    if (N > SKINNY_MAX_WIDTH || K > SKINNY_MAX_WIDTH) return SKINNY_ERR_UNSUPPORTED;
    return SKINNY_OK;
}

bool rows16(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// Whether rows of wa and wb bytes, the second b - a = `apart` behind the first and both every `step` bytes, share none.
bool beside(uintptr_t apart, int64_t step, int64_t wa, int64_t wb) {
    int64_t d = (int64_t)apart % step;
    if (d < 0) d += step;
    return wa <= step && wb <= step && d >= wa && d + wb <= step;
}
// The bytes of a matrix, and its rows' distance and width (one row or a plain range: 0).
struct Rows : Range {
    int64_t step = 0, width = 0;
};
Rows rows_of(const void *p, int64_t rows, int64_t cols, int64_t ld, int el) {
    const Range r = span(p, rows, cols, ld, el);
    return {r, rows > 1 ? ld * el : 0, cols * el};
}
// Whether a matrix that is written shares elements with one of the others; columns of one buffer side by side do not.
bool rows_meet(const Rows &w, std::initializer_list<Rows> others) {
    for (const Rows &o : others)
        if (meets(w, {o}) && !(w.step > 0 && w.step == o.step && beside(o.lo - w.lo, w.step, w.width, o.width))) return true;
    return false;
}

// Where the pieces of a call lie in its workspace (-1: not used).
struct Space {
    int64_t x = -1, w = -1, dz = -1, partial = -1, bytes = 0;
    int64_t take(int64_t n) {
        const int64_t at = bytes;
        bytes += pad16(n);
        return at;
    }
};
Space linear_space(const void *X, int ldx, const void *W, int ldw, int M, int K, int rows) {
    Space s;
    if (K == 0) return s;
    if (!rows16(X, ldx)) s.x = s.take((int64_t)M * pad8(K) * 2);
    if (!rows16(W, ldw)) s.w = s.take((int64_t)rows * pad8(K) * 2);
    return s;
}
// dZ (or dY on 16-byte boundaries), X and W likewise, the parts of the bias gradient
Space grad_space(const void *dY, int lddy, const void *X, int ldx, const void *W, int ldw, int M, int K, int rows, int act) {
    Space s;
    if (act != SKINNY_ACT_NONE || !rows16(dY, lddy)) s.dz = s.take((int64_t)M * pad8(rows) * 2);
    if (!rows16(X, ldx)) s.x = s.take((int64_t)M * pad8(K) * 2);
    if (!rows16(W, ldw)) s.w = s.take((int64_t)rows * pad8(K) * 2);
    s.partial = s.take((int64_t)kDbiasParts * rows * 4);
    return s;
}

skinny_status_t launch_product(const ProductArgs &a, const CallCtx &c, cudaStream_t s) {
    if (a.depth == 0) return launched(launch_linear_empty(a, c, s));
    const bool pair = c.force_backend == SKINNY_BACKEND_TCGEN05 ||
                      (c.force_backend != SKINNY_BACKEND_SPLITK && linear_pair_faster(a, c.num_sms));
    return launched(pair ? launch_linear_pair(a, c, s) : launch_linear_tc(a, c, s));
}

// [T, H] rows of D elements, strides st and sh.
struct View {
    const void *p;
    int64_t st, sh;
    int T, H, D, el;
    bool none() const { return !p || T == 0 || H == 0; }
    bool ok() const {      // heads do not overlap
        if (T <= 1 && H <= 1) return true;
        const int64_t s = T > 1 ? st : INT64_MAX, h = H > 1 ? sh : INT64_MAX;
        if (s < D || h < D) return false;
        if (T <= 1 || H <= 1) return true;
        return st - D >= (H - 1) * sh || (sh - D) / (T - 1) >= st;
    }
    int64_t extent() const { return ((T - 1) * (T > 1 ? st : 0) + (H - 1) * (H > 1 ? sh : 0) + D) * el; }
    bool same(const View &o) const {
        return p == o.p && T == o.T && H == o.H && (T <= 1 || st == o.st) && (H <= 1 || sh == o.sh);
    }
};
bool views_meet(const View &a, const View &b) {
    if (a.none() || b.none()) return false;
    const uintptr_t a0 = addr(a.p), b0 = addr(b.p);
    if (!ranges_overlap(a0, a0 + (uintptr_t)a.extent(), b0, b0 + (uintptr_t)b.extent())) return false;
    // side by side in rows of one stride: neither reaches into the other within a row
    const int64_t s = a.st * a.el, wa = ((int64_t)(a.H - 1) * (a.H > 1 ? a.sh : 0) + a.D) * a.el,
                  wb = ((int64_t)(b.H - 1) * (b.H > 1 ? b.sh : 0) + b.D) * b.el;
    if (a.T > 1 && b.T > 1 && a.st == b.st && beside(b0 - a0, s, wa, wb)) return false;
    // heads by turns, a query's beside its key's: all strides are multiples of one, and the heads lie at different
    // places of it
    int64_t step = 0;
    for (const View *v : {&a, &b})
        for (int64_t m : {v->T > 1 ? v->st : 0, v->H > 1 ? v->sh : 0})
            if (m && (!step || m < step)) step = m;
    for (const View *v : {&a, &b})
        if (step && ((v->T > 1 && v->st % step) || (v->H > 1 && v->sh % step))) step = 0;
    return !(step && beside(b0 - a0, step * a.el, (int64_t)a.D * a.el, (int64_t)b.D * b.el));
}
bool view_meets_range(const View &a, const Range &r) {
    if (a.none() || r.lo >= r.hi) return false;
    return ranges_overlap(addr(a.p), addr(a.p) + (uintptr_t)a.extent(), r.lo, r.hi);
}

constexpr int64_t kMaxStride = 1ll << 40, kMaxExtent = 1ll << 48;      // elements

// What both directions ask of their arguments.
skinny_status_t check_heads(const skinny_heads_t *q, const skinny_heads_t *k, const skinny_rotation_t *rot, int T, int D,
                            int norm, int dtype) {
    if (!q || !k || !rot || T < 0 || D < 1 || !dtype_ok(dtype) || q->H < 0 || k->H < 0) return SKINNY_ERR_INVALID_VALUE;
    if (D > SKINNY_MAX_HEAD || rot->axes > SKINNY_MAX_AXES || q->H > SKINNY_MAX_WIDTH || k->H > SKINNY_MAX_WIDTH)
        return SKINNY_ERR_UNSUPPORTED;
    if (rot->R < 0 || rot->R > D || rot->R % 2) return SKINNY_ERR_INVALID_VALUE;
    if (rot->R > 0) {
        if (rot->axes < 1 || rot->P < 1 || (T > 0 && (!rot->table || !rot->positions))) return SKINNY_ERR_INVALID_VALUE;
        if (!aligned(rot->table, 4) || !aligned(rot->positions, 4) || !aligned(rot->pair_axis, 4)) return SKINNY_ERR_MISALIGNED;
    }
    for (const skinny_heads_t *h : {q, k})
        if (norm && h->H > 0 && !aligned(h->w, el_bytes(dtype))) return SKINNY_ERR_MISALIGNED;
    return SKINNY_OK;
}
skinny_status_t check_view(const View &v) {
    if (v.T == 0 || v.H == 0) return SKINNY_OK;
    if (!v.p || v.st < 0 || v.sh < 0 || v.st > kMaxStride || v.sh > kMaxStride || !v.ok()) return SKINNY_ERR_INVALID_VALUE;
    if ((v.T > 1 && v.st > kMaxExtent / v.T) || (v.H > 1 && v.sh > kMaxExtent / v.H)) return SKINNY_ERR_INVALID_VALUE;
    return aligned(v.p, v.el) ? SKINNY_OK : SKINNY_ERR_MISALIGNED;
}
// Whether what is written meets the small inputs.
bool meets_tables(const View &v, const skinny_heads_t *q, const skinny_heads_t *k, const skinny_rotation_t *rot, int T,
                  int D, int norm) {
    const int64_t R = rot->R;
    for (const skinny_heads_t *h : {q, k})
        if (norm && h->H > 0 && view_meets_range(v, span(h->w, 1, D, D, v.el))) return true;
    if (R == 0) return false;
    return view_meets_range(v, span(rot->table, rot->P, R, R, 4)) ||
           view_meets_range(v, span(rot->positions, rot->axes, T, T, 4)) ||
           view_meets_range(v, span(rot->pair_axis, 1, R / 2, R / 2, 4));
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

int64_t skinny_linear_workspace(const uint16_t *X, int ldx, const uint16_t *W, int ldw, int M, int N, int K, int act) {
    if (check_product(M, N, K, act) != SKINNY_OK || M == 0 || N == 0) return 0;
    return linear_space(X, ldx, W, ldw, M, K, act_gated(act) ? 2 * N : N).bytes;
}

skinny_status_t skinny_linear_bf16(const uint16_t *X, int ldx, const uint16_t *W, int ldw, const uint16_t *bias,
                                   const void *R, int ldr, void *Y, int ldy, uint16_t *Z, int ldz, int M, int N, int K,
                                   int act, int out_dtype, void *workspace, int64_t workspace_bytes, void *stream) {
    skinny_status_t st = check_product(M, N, K, act);
    if (st != SKINNY_OK) return st;
    if (!dtype_ok(out_dtype)) return SKINNY_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return SKINNY_OK;
    const int rows = act_gated(act) ? 2 * N : N, ob = el_bytes(out_dtype);
    const int64_t need = skinny_linear_workspace(X, ldx, W, ldw, M, N, K, act);
    if (!Y || ldy < N || (R && ldr < N) || (Z && ldz < rows) || (K > 0 && (!X || !W || ldx < K || ldw < K)) ||
        (need > 0 && (!workspace || workspace_bytes < need)))
        return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(Y, ob) || !aligned(R, ob) || !aligned(Z, 2) || !aligned(bias, 2) ||
        (K > 0 && (!aligned(X, 2) || !aligned(W, 2))) || (need > 0 && !aligned(workspace, 16)))
        return SKINNY_ERR_MISALIGNED;
    const Rows none{}, y = rows_of(Y, M, N, ldy, ob), z = rows_of(Z, M, rows, ldz, 2), b = rows_of(bias, 1, rows, rows, 2),
               x = K > 0 ? rows_of(X, M, K, ldx, 2) : none, w = K > 0 ? rows_of(W, rows, K, ldw, 2) : none,
               r = rows_of(R, M, N, ldr, ob), ws = {{addr(workspace), addr(workspace) + (uintptr_t)need}};
    const bool in_place = R == Y && (M == 1 || ldr == ldy);
    if (rows_meet(y, {x, w, b, z, ws}) || (!in_place && rows_meet(y, {r})) || rows_meet(z, {x, w, b, r, ws}) ||
        rows_meet(ws, {x, w, b, r}))
        return SKINNY_ERR_INVALID_VALUE;
    CallCtx c;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProductArgs a{{W, ldw, false}, {X, ldx, false}, M, N, K, act, bias, R, ldr, Y, ldy, Z, ldz, out_dtype == SKINNY_BF16,
                  false, true};
    const Space sp = linear_space(X, ldx, W, ldw, M, K, rows);
    if (sp.bytes > 0) {
        uint8_t *space = static_cast<uint8_t *>(workspace);
        PackArgs px{}, pw{};
        if (sp.x >= 0) {
            px = {X, ldx, M, K, reinterpret_cast<uint16_t *>(space + sp.x)};
            a.B = {px.to, pad8(K), false};
        }
        if (sp.w >= 0) {
            pw = {W, ldw, rows, K, reinterpret_cast<uint16_t *>(space + sp.w)};
            a.A = {pw.to, pad8(K), false};
        }
        if (launch_rows_pack(px, pw, c, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
    }
    return launch_product(a, c, s);
}

int64_t skinny_linear_grad_workspace(const uint16_t *dY, int lddy, const uint16_t *X, int ldx, const uint16_t *W, int ldw,
                                     int M, int N, int K, int act) {
    if (check_product(M, N, K, act) != SKINNY_OK || M == 0 || N == 0) return 0;
    return grad_space(dY, lddy, X, ldx, W, ldw, M, K, act_gated(act) ? 2 * N : N, act).bytes;
}

skinny_status_t skinny_linear_grad_bf16(const uint16_t *dY, int lddy, const uint16_t *X, int ldx, const uint16_t *W,
                                        int ldw, const uint16_t *Z, int ldz, uint16_t *dX, int lddx, uint16_t *dW,
                                        int lddw, float *dbias, int M, int N, int K, int act, void *workspace,
                                        int64_t workspace_bytes, void *stream) {
    skinny_status_t st = check_product(M, N, K, act);
    if (st != SKINNY_OK) return st;
    const int rows = act_gated(act) ? 2 * N : N;
    if (K == 0) dX = dW = nullptr;
    if (M == 0) dX = nullptr;
    if (N == 0) { dW = nullptr; dbias = nullptr; }
    if (!dX && !dW && !dbias) return SKINNY_OK;
    if ((dX && lddx < K) || (dW && lddw < K)) return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(dX, 2) || !aligned(dW, 2) || !aligned(dbias, 4)) return SKINNY_ERR_MISALIGNED;
    const Rows none{}, gx = rows_of(dX, M, K, lddx, 2), gw = rows_of(dW, rows, K, lddw, 2), gb = rows_of(dbias, 1, rows, rows, 4);
    if (rows_meet(gx, {gw, gb}) || rows_meet(gw, {gb})) return SKINNY_ERR_INVALID_VALUE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallCtx c;
    if (M == 0 || N == 0) {          // empty sums
        st = call_context(&c);
        if (st != SKINNY_OK) return st;
        if (dX && cudaMemset2DAsync(dX, (size_t)lddx * 2, 0, (size_t)K * 2, (size_t)M, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
        if (dW && cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)K * 2, (size_t)rows, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)rows * 4, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
        return SKINNY_OK;
    }
    const bool act_none = act == SKINNY_ACT_NONE;
    const int64_t need = skinny_linear_grad_workspace(dY, lddy, X, ldx, W, ldw, M, N, K, act);
    if (!dY || lddy < N || (!act_none && (!Z || ldz < rows)) || (dX && (!W || ldw < K)) || (dW && (!X || ldx < K)) ||
        !workspace || workspace_bytes < need)
        return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(dY, 2) || (!act_none && !aligned(Z, 2)) || (dX && !aligned(W, 2)) || (dW && !aligned(X, 2)) ||
        !aligned(workspace, 16))
        return SKINNY_ERR_MISALIGNED;
    const Rows y = rows_of(dY, M, N, lddy, 2), z = act_none ? none : rows_of(Z, M, rows, ldz, 2),
               x = dW ? rows_of(X, M, K, ldx, 2) : none, w = dX ? rows_of(W, rows, K, ldw, 2) : none,
               ws = {{addr(workspace), addr(workspace) + (uintptr_t)need}};
    if (rows_meet(gx, {y, z, x, w, ws}) || rows_meet(gw, {y, z, x, w, ws}) || rows_meet(gb, {y, z, x, w, ws}) ||
        rows_meet(ws, {y, z, x, w}))
        return SKINNY_ERR_INVALID_VALUE;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    const Space sp = grad_space(dY, lddy, X, ldx, W, ldw, M, K, rows, act);
    uint8_t *space = static_cast<uint8_t *>(workspace);
    Operand dz{dY, lddy, false}, xo{X, ldx, true}, wo{W, ldw, true};
    bool beside = false;             // the next kernel needs nothing of the one before
    if (dX || dW) {
        PackArgs px{}, pw{};
        if (dW && sp.x >= 0) {
            px = {X, ldx, M, K, reinterpret_cast<uint16_t *>(space + sp.x)};
            xo = {px.to, pad8(K), true};
        }
        if (dX && sp.w >= 0) {
            pw = {W, ldw, rows, K, reinterpret_cast<uint16_t *>(space + sp.w)};
            wo = {pw.to, pad8(K), true};
        }
        if (launch_rows_pack(px, pw, c, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
        beside = px.from || pw.from;
    }
    if (dbias || ((dX || dW) && sp.dz >= 0)) {
        uint16_t *to = sp.dz >= 0 && (dX || dW) ? reinterpret_cast<uint16_t *>(space + sp.dz) : nullptr;
        const LinearDzArgs d{dY, lddy, act_none ? nullptr : Z, ldz, to, pad8(rows), dbias,
                             reinterpret_cast<float *>(space + sp.partial), M, N, act, beside};
        if (launch_linear_dz(d, c, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
        if (to) dz = {to, pad8(rows), false};
        beside = dbias && dbias_parts(M) > 1;        // the products do not read the bias gradient
    } else {
        beside = false;                              // but the rows laid out
    }
    if (dX) {
        const ProductArgs a{wo, dz, M, K, rows, SKINNY_ACT_NONE, nullptr, nullptr, 0, dX, lddx, nullptr, 0, 1,
                            beside, !dW};
        st = launch_product(a, c, s);
        if (st != SKINNY_OK) return st;
    }
    if (dW) {
        const ProductArgs a{xo, {dz.p, dz.ld, true}, rows, K, M, SKINNY_ACT_NONE, nullptr, nullptr, 0, dW, lddw, nullptr, 0,
                            1, beside || dX, true};
        st = launch_product(a, c, s);
        if (st != SKINNY_OK) return st;
    }
    return SKINNY_OK;
}

skinny_status_t skinny_qk_norm_rope(const skinny_heads_t *q, const skinny_heads_t *k, const skinny_rotation_t *rot, int T,
                                    int D, int norm, float eps, int dtype, void *q_out, int64_t q_st, int64_t q_sh,
                                    void *k_out, int64_t k_st, int64_t k_sh, void *stream) {
    skinny_status_t st = check_heads(q, k, rot, T, D, norm, dtype);
    if (st != SKINNY_OK) return st;
    if (T == 0 || (q->H == 0 && k->H == 0)) return SKINNY_OK;
    const int el = el_bytes(dtype);
    const View in[2] = {{q->x, q->st, q->sh, T, q->H, D, el}, {k->x, k->st, k->sh, T, k->H, D, el}},
               out[2] = {{q_out, q_st, q_sh, T, q->H, D, el}, {k_out, k_st, k_sh, T, k->H, D, el}};
    for (const View &v : {in[0], in[1], out[0], out[1]}) {
        st = check_view(v);
        if (st != SKINNY_OK) return st;
    }
    if (views_meet(out[0], out[1])) return SKINNY_ERR_INVALID_VALUE;
    for (int i = 0; i < 2; ++i) {
        if (out[i].H == 0) continue;
        if ((!out[i].same(in[i]) && views_meet(out[i], in[i])) || views_meet(out[i], in[1 - i]) ||
            meets_tables(out[i], q, k, rot, T, D, norm))
            return SKINNY_ERR_INVALID_VALUE;
    }
    CallCtx c;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    HeadsArgs a{};
    a.side[0] = {q->x, q->st, q->sh, q->w, nullptr, 0, 0, q_out, q_st, q_sh, nullptr, q->H};
    a.side[1] = {k->x, k->st, k->sh, k->w, nullptr, 0, 0, k_out, k_st, k_sh, nullptr, k->H};
    a.table = rot->table; a.P = rot->P; a.positions = rot->positions; a.pair_axis = rot->pair_axis;
    a.axes = rot->axes; a.R = rot->R; a.interleaved = rot->interleaved;
    a.T = T; a.D = D; a.norm = norm != 0; a.eps = eps; a.b16 = dtype == SKINNY_BF16;
    return launched(launch_heads(a, c, static_cast<cudaStream_t>(stream)));
}

int64_t skinny_qk_norm_rope_grad_workspace(int T, int q_heads, int k_heads, int D) {
    if (T < 0 || q_heads < 0 || k_heads < 0 || D < 1 || D > SKINNY_MAX_HEAD) return 0;
    const int64_t heads = (int64_t)T * ((int64_t)q_heads + k_heads);      // a CTA has one at least
    return (heads < kHeadsParts ? heads : kHeadsParts) * 2 * D * 4;
}

skinny_status_t skinny_qk_norm_rope_grad(const void *dq, int64_t dq_st, int64_t dq_sh, const void *dk, int64_t dk_st,
                                         int64_t dk_sh, const skinny_heads_t *q, const skinny_heads_t *k,
                                         const skinny_rotation_t *rot, int T, int D, int norm, float eps, int dtype,
                                         void *q_grad, int64_t qg_st, int64_t qg_sh, void *k_grad, int64_t kg_st,
                                         int64_t kg_sh, float *q_wgrad, float *k_wgrad, void *workspace,
                                         int64_t workspace_bytes, void *stream) {
    skinny_status_t st = check_heads(q, k, rot, T, D, norm, dtype);
    if (st != SKINNY_OK) return st;
    if (!norm && (q_wgrad || k_wgrad)) return SKINNY_ERR_INVALID_VALUE;
    if (!aligned(q_wgrad, 4) || !aligned(k_wgrad, 4)) return SKINNY_ERR_MISALIGNED;
    const bool sums = q_wgrad || k_wgrad;
    const Range wq = span(q_wgrad, 1, D, D, 4), wk = span(k_wgrad, 1, D, D, 4);
    if (meets(wq, {wk})) return SKINNY_ERR_INVALID_VALUE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallCtx c;
    if (T == 0 || (q->H == 0 && k->H == 0)) {          // empty sums
        if (!sums) return SKINNY_OK;
        st = call_context(&c);
        if (st != SKINNY_OK) return st;
        for (float *w : {q_wgrad, k_wgrad})
            if (w && cudaMemsetAsync(w, 0, (size_t)D * 4, s) != cudaSuccess) return SKINNY_ERR_LAUNCH;
        return SKINNY_OK;
    }
    const int el = el_bytes(dtype);
    const int64_t need = sums ? skinny_qk_norm_rope_grad_workspace(T, q->H, k->H, D) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return SKINNY_ERR_INVALID_VALUE;
    if (need > 0 && !aligned(workspace, 16)) return SKINNY_ERR_MISALIGNED;
    const Range ws = {addr(workspace), addr(workspace) + (uintptr_t)need};
    const View x[2] = {{q->x, q->st, q->sh, T, q->H, D, el}, {k->x, k->st, k->sh, T, k->H, D, el}},
               d[2] = {{dq, dq_st, dq_sh, T, q->H, D, el}, {dk, dk_st, dk_sh, T, k->H, D, el}},
               y[2] = {{q_grad, qg_st, qg_sh, T, q->H, D, el}, {k_grad, kg_st, kg_sh, T, k->H, D, el}};
    for (const View &v : {d[0], d[1], y[0], y[1]}) {
        st = check_view(v);
        if (st != SKINNY_OK) return st;
    }
    for (int i = 0; norm && i < 2; ++i) {
        st = check_view(x[i]);
        if (st != SKINNY_OK) return st;
    }
    if (views_meet(y[0], y[1])) return SKINNY_ERR_INVALID_VALUE;
    for (int i = 0; i < 2; ++i) {
        if (y[i].H == 0) continue;
        if ((!y[i].same(d[i]) && views_meet(y[i], d[i])) || views_meet(y[i], d[1 - i]) ||
            (norm && (views_meet(y[i], x[0]) || views_meet(y[i], x[1]))) || meets_tables(y[i], q, k, rot, T, D, norm) ||
            view_meets_range(y[i], ws) || view_meets_range(y[i], wq) || view_meets_range(y[i], wk))
            return SKINNY_ERR_INVALID_VALUE;
    }
    // the sums and their workspace against every input
    for (const Range &w : {wq, wk, ws}) {
        if (w.lo >= w.hi) continue;
        const View v{reinterpret_cast<const void *>(w.lo), 0, 0, 1, 1, (int)((w.hi - w.lo) / el), el};
        if (views_meet(v, x[0]) || views_meet(v, x[1]) || views_meet(v, d[0]) || views_meet(v, d[1]) ||
            meets_tables(v, q, k, rot, T, D, norm))
            return SKINNY_ERR_INVALID_VALUE;
    }
    if (meets(ws, {wq, wk})) return SKINNY_ERR_INVALID_VALUE;
    st = call_context(&c);
    if (st != SKINNY_OK) return st;
    HeadsArgs a{};
    a.side[0] = {q->x, q->st, q->sh, q->w, dq, dq_st, dq_sh, q_grad, qg_st, qg_sh, q_wgrad, q->H};
    a.side[1] = {k->x, k->st, k->sh, k->w, dk, dk_st, dk_sh, k_grad, kg_st, kg_sh, k_wgrad, k->H};
    a.table = rot->table; a.P = rot->P; a.positions = rot->positions; a.pair_axis = rot->pair_axis;
    a.axes = rot->axes; a.R = rot->R; a.interleaved = rot->interleaved;
    a.T = T; a.D = D; a.norm = norm != 0; a.eps = eps; a.b16 = dtype == SKINNY_BF16; a.grad = true;
    a.partial = static_cast<float *>(workspace);
    return launched(launch_heads(a, c, s));
}

}  // extern "C"
