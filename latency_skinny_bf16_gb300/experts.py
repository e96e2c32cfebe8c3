"""Around the router and the decode projections of a mixture-of-experts layer:
tokens sorted by expert and back with their gradients, the experts' products,
and a shared projection with a low-rank adapter per token.

As in the package itself, the ``skinny_*`` functions carry the C names of
``include/skinny_experts.h`` and only marshal arguments; the tensor functions
(:func:`expert_dispatch`, :func:`expert_combine`, :func:`expert_combine_grad`,
:func:`experts_gemm`, :func:`lora_gemm`) take CUDA tensors, allocate what is
not given on the stream they launch on, and raise on a refusal.
"""
from __future__ import annotations

import ctypes

import latency_skinny_bf16_gb300 as _sk

SKINNY_BF16 = 0
SKINNY_F32 = 1
SKINNY_ACT_NONE = 0
SKINNY_ACT_SWIGLU = 1
SKINNY_MAX_TOPK = 64
SKINNY_MAX_SORT_EXPERTS = 8192
SKINNY_MAX_EXPERTS = 1024
SKINNY_MAX_RANK = 256
SKINNY_MAX_WIDTH = 1 << 20

__all__ = [
    "SKINNY_BF16", "SKINNY_F32", "SKINNY_ACT_NONE", "SKINNY_ACT_SWIGLU", "SKINNY_MAX_TOPK", "SKINNY_MAX_SORT_EXPERTS",
    "SKINNY_MAX_EXPERTS", "SKINNY_MAX_RANK", "SKINNY_MAX_WIDTH",
    "skinny_expert_dispatch", "skinny_expert_combine", "skinny_expert_combine_grad",
    "skinny_experts_gemm_bf16", "skinny_lora_gemm_bf16", "skinny_lora_workspace",
    "expert_dispatch", "expert_combine", "expert_combine_grad", "experts_gemm", "lora_gemm", "lora_workspace",
]

_fits_int = _sk._fits_int
_ACTS = {"none": SKINNY_ACT_NONE, None: SKINNY_ACT_NONE, "swiglu": SKINNY_ACT_SWIGLU}

SYMBOLS = ("skinny_expert_dispatch", "skinny_expert_combine", "skinny_expert_combine_grad", "skinny_experts_gemm_bf16",
           "skinny_lora_gemm_bf16", "skinny_lora_workspace")


def bind(lib: ctypes.CDLL) -> None:
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.skinny_expert_dispatch.argtypes = [vp, i, vp, i, i, i, i, i, i, vp, vp, vp, vp, i, vp]
    lib.skinny_expert_combine.argtypes = [vp, i, i, vp, vp, i, i, i, i, i, i, vp, i, vp]
    lib.skinny_expert_combine_grad.argtypes = [vp, i, vp, i, i, vp, vp, i, i, i, i, i, vp, i, vp, i, vp]
    ll = ctypes.c_int64
    lib.skinny_experts_gemm_bf16.argtypes = [vp, i, i, vp, vp, i, ll, i, i, i, i, i, vp, i, vp]
    lib.skinny_lora_gemm_bf16.argtypes = [vp, i, vp, i, vp, i, ll, vp, i, ll, vp, vp, vp, i, i, vp, i, i, i, i, i, vp,
                                          ll, vp]
    lib.skinny_lora_workspace.argtypes = [i, i, i, i]
    for name in SYMBOLS:
        getattr(lib, name).restype = i
    lib.skinny_lora_workspace.restype = ll


_loaded = None


def _lib() -> ctypes.CDLL:
    global _loaded
    if _loaded is None:
        _loaded = _sk.load_library()
    return _loaded


# ---------------------------------------------------------------- C-named wrappers (raw pointers)

def skinny_expert_dispatch(ids: int, ldid: int, X: int, ldx: int, T: int, k: int, E: int, H: int, dtype: int,
                           pos: int, order: int, offsets: int, Xs: int, ldxs: int, stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_expert_dispatch(ids, ldid, X, ldx, T, k, E, H, dtype, pos, order, offsets, Xs,
                                                     ldxs, stream)


def skinny_expert_combine(Ys: int, ldys: int, rows: int, pos: int, weights: int, ldw: int, T: int, k: int, H: int,
                          in_dtype: int, out_dtype: int, Y: int, ldy: int, stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_expert_combine(Ys, ldys, rows, pos, weights, ldw, T, k, H, in_dtype, out_dtype,
                                                    Y, ldy, stream)


def skinny_expert_combine_grad(dY: int, lddy: int, Ys: int, ldys: int, rows: int, pos: int, weights: int, ldw: int,
                               T: int, k: int, H: int, dtype: int, dYs: int, lddys: int, dweights: int, lddw: int,
                               stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_expert_combine_grad(dY, lddy, Ys, ldys, rows, pos, weights, ldw, T, k, H, dtype,
                                                         dYs, lddys, dweights, lddw, stream)


def skinny_experts_gemm_bf16(Xs: int, ldx: int, rows: int, offsets: int, W: int, ldw: int, ldwe: int, E: int, N: int,
                             K: int, act: int, out_dtype: int, Y: int, ldy: int, stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_experts_gemm_bf16(Xs, ldx, rows, offsets, W, ldw, ldwe, E, N, K, act, out_dtype,
                                                       Y, ldy, stream)


def skinny_lora_gemm_bf16(X: int, ldx: int, W: int, ldw: int, A: int, lda: int, ldae: int, B: int, ldb: int,
                          ldbe: int, adapters: int, ranks: int, scales: int, L: int, R: int, Y: int, ldy: int, M: int,
                          N: int, K: int, out_dtype: int, workspace: int, workspace_bytes: int,
                          stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_lora_gemm_bf16(X, ldx, W, ldw, A, lda, ldae, B, ldb, ldbe, adapters, ranks,
                                                    scales, L, R, Y, ldy, M, N, K, out_dtype, workspace,
                                                    workspace_bytes, stream)


def skinny_lora_workspace(M: int, N: int, R: int, out_dtype: int) -> int:
    """Bytes of workspace of skinny_lora_gemm_bf16; 0 for sizes it refuses."""
    return _lib().skinny_lora_workspace(M, N, R, out_dtype)


# ---------------------------------------------------------------- tensors

torch = None    # imported by the first call that takes tensors: the C-named functions need none


def _import_torch():
    global torch, _current
    import torch
    if hasattr(torch._C, "_cuda_getCurrentRawStream"):
        # the same handle without a Stream object
        def _current(device):
            return torch._C._cuda_getCurrentRawStream(device.index)


def _dtype(t, name):
    d = t.dtype
    if d is torch.bfloat16:
        return SKINNY_BF16
    if d is torch.float32:
        return SKINNY_F32
    raise TypeError(f"{name} must be bfloat16 or float32, not {d}")


def _rows(t, name, dtype=None):
    """(rows, columns, row stride) of a CUDA matrix with unit column stride."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA matrix, not {tuple(shape)} on {t.device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    m, n = shape
    ld, one = t.stride()
    if n > 1 and one != 1:
        raise ValueError(f"{name} needs unit column stride")
    if m <= 1:
        ld = n or 1
    elif ld < n:
        raise ValueError(f"{name} needs rows that do not overlap")
    if (m | ld) >> 31:          # n <= ld
        _fits_int(name, m, ld)
    return m, n, ld


def _flat(t, name, n, dtype):
    """Address of a contiguous CUDA tensor of n elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} elements")
    return t.data_ptr()


def _on(stream, device):
    """The context of a given stream: inside it is torch's current one, so what
    a call allocates belongs to it."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _current(device):
    """Handle of torch's current stream."""
    return torch.cuda.current_stream(device).cuda_stream


def _refused(st, what):
    raise _sk.SkinnyError(st, what)


def expert_dispatch(ids, num_experts, x=None, xs=None, pos=None, order=None, offsets=None, stream=None):
    """Tokens sorted by expert: for the router's ``ids`` int32 [T, k] (an id
    outside ``[0, num_experts)`` drops the entry) returns ``(xs, pos, order,
    offsets)``: ``xs`` [T*k, H] with ``x``'s rows in expert order (rows from
    ``offsets[num_experts]`` on are left as they are; None without ``x``),
    ``pos`` int32 [T, k] (-1: dropped), ``order`` int32 [T*k], ``offsets``
    int32 [num_experts + 1].  See ``skinny_expert_dispatch``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _on(stream, ids.device):
            return expert_dispatch(ids, num_experts, x, xs, pos, order, offsets)
    T, k, ldid = _rows(ids, "ids", torch.int32)
    if num_experts >> 31:
        _fits_int("num_experts", num_experts)
    n, dev = T * k, ids.device
    if pos is None:
        pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    if order is None:
        order = torch.empty(n, dtype=torch.int32, device=dev)
    if offsets is None:
        offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    pp, op = _flat(pos, "pos", n, torch.int32), _flat(order, "order", n, torch.int32)
    fp = _flat(offsets, "offsets", num_experts + 1, torch.int32)
    if x is None:
        xp = sp = ldx = ldxs = H = dt = 0
    else:
        xrows, H, ldx = _rows(x, "x")
        dt = _dtype(x, "x")
        if xrows != T:
            raise ValueError(f"x has {xrows} rows, ids {T}")
        if xs is None:
            xs = torch.empty((n, H), dtype=x.dtype, device=dev)
        srows, scols, ldxs = _rows(xs, "xs", x.dtype)
        if srows != n or scols != H:
            raise ValueError(f"xs must be {(n, H)}, not {tuple(xs.shape)}")
        xp, sp = x.data_ptr(), xs.data_ptr()
    st = _lib().skinny_expert_dispatch(ids.data_ptr(), ldid, xp, ldx, T, k, num_experts, H, dt, pp, op, fp, sp, ldxs,
                                       _current(dev))
    if st:
        _refused(st, "skinny_expert_dispatch")
    return xs, pos, order, offsets


def _weights(weights, T, k):
    if weights is None:
        return 0, 0
    m, n, ld = _rows(weights, "weights", torch.float32)
    if m != T or n != k:
        raise ValueError(f"weights must be {(T, k)}, not {(m, n)}")
    return weights.data_ptr(), ld


def _pos(pos):
    shape = pos.shape
    if len(shape) != 2:
        raise ValueError(f"pos must be [T, k], not {tuple(shape)}")
    T, k = shape
    if (T | k) >> 31:
        _fits_int("pos", T, k)
    return T, k, _flat(pos, "pos", T * k, torch.int32)


def expert_combine(ys, pos, weights=None, out=None, stream=None):
    """``out[t] = sum_j weights[t, j] * ys[pos[t, j]]`` over the live entries
    (``0 <= pos < ys.shape[0]``), summed in fp32: ``ys`` bf16 or fp32 [rows,
    H], ``pos`` int32 [T, k] from :func:`expert_dispatch`, ``weights`` fp32
    [T, k] or None (ones: the gradient of dispatch's copies), ``out`` bf16 or
    fp32 [T, H] (default: as ``ys``).  See ``skinny_expert_combine``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _on(stream, ys.device):
            return expert_combine(ys, pos, weights, out)
    rows, H, ldys = _rows(ys, "ys")
    it = _dtype(ys, "ys")
    T, k, pp = _pos(pos)
    wp, ldw = _weights(weights, T, k)
    if out is None:
        out = torch.empty((T, H), dtype=ys.dtype, device=ys.device)
    orows, ocols, ldy = _rows(out, "out")
    if orows != T or ocols != H:
        raise ValueError(f"out must be {(T, H)}, not {(orows, ocols)}")
    st = _lib().skinny_expert_combine(ys.data_ptr(), ldys, rows, pp, wp, ldw, T, k, H, it, _dtype(out, "out"),
                                      out.data_ptr(), ldy, _current(ys.device))
    if st:
        _refused(st, "skinny_expert_combine")
    return out


def expert_combine_grad(dy, ys, pos, weights=None, dys=None, dweights=None, stream=None, weight_grad=True):
    """The gradient of :func:`expert_combine` for ``dy`` [T, H]: returns
    ``(dys, dweights)`` with ``dys[pos[t, j]] = weights[t, j] * dy[t]`` (the
    type of ``dy``; rows no entry names are left as they are) and
    ``dweights[t, j] = <dy[t], ys[pos[t, j]]>`` (fp32; 0 for a dropped entry).
    ``weight_grad=False`` (a router that is not trained) leaves dweights out
    and reads nothing of ``ys``, which then only gives the number of rows.  See
    ``skinny_expert_combine_grad``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _on(stream, dy.device):
            return expert_combine_grad(dy, ys, pos, weights, dys, dweights, None, weight_grad)
    T, H, lddy = _rows(dy, "dy")
    dt = _dtype(dy, "dy")
    rows, ycols, ldys = _rows(ys, "ys", dy.dtype)
    prows, k, pp = _pos(pos)
    if prows != T or ycols != H:
        raise ValueError(f"shape mismatch: dy {tuple(dy.shape)}, ys {tuple(ys.shape)}, pos {tuple(pos.shape)}")
    wp, ldw = _weights(weights, T, k)
    if dys is None:
        dys = torch.empty((rows, H), dtype=dy.dtype, device=dy.device)
    grows, gcols, lddys = _rows(dys, "dys", dy.dtype)
    dwp, wrows, wcols, lddw = 0, T, k, 0
    if weight_grad:
        if dweights is None:
            dweights = torch.empty((T, k), dtype=torch.float32, device=dy.device)
        wrows, wcols, lddw = _rows(dweights, "dweights", torch.float32)
        dwp = dweights.data_ptr()
    elif dweights is not None:
        raise ValueError("dweights is given, and weight_grad is False")
    if grows != rows or gcols != H or wrows != T or wcols != k:
        raise ValueError(f"dys must be {(rows, H)} and dweights {(T, k)}")
    st = _lib().skinny_expert_combine_grad(dy.data_ptr(), lddy, ys.data_ptr(), ldys, rows, pp, wp, ldw, T, k, H, dt,
                                           dys.data_ptr(), lddys, dwp, lddw, _current(dy.device))
    if st:
        _refused(st, "skinny_expert_combine_grad")
    return dys, dweights


def _stack(t, name, rows, cols):
    """(row stride, matrix stride) of a CUDA bf16 stack of matrices [n, rows, cols]."""
    shape = t.shape
    if len(shape) != 3 or not t.is_cuda or t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor of three dimensions")
    n, r, c = shape
    if r != rows or c != cols:
        raise ValueError(f"{name} must hold {rows} x {cols} matrices, not {r} x {c}")
    lde, ld, one = t.stride()
    if c > 1 and one != 1:
        raise ValueError(f"{name} needs unit stride along its last dimension")
    if r <= 1:
        ld = c or 1
    if (n | r | ld) >> 31:
        _fits_int(name, n, r, ld)
    return ld, lde if n > 1 else (r or 1) * ld


def experts_gemm(xs, offsets, w, out=None, activation=None, stream=None):
    """The experts' products on rows in expert order: ``out[r] = xs[r] .
    w[e]^T`` for ``offsets[e] <= r < offsets[e+1]``, ``xs`` bf16 [rows, K],
    ``offsets`` int32 [E+1] from :func:`expert_dispatch`, ``w`` bf16 [E, N, K].
    ``activation="swiglu"``: ``w`` is [E, 2N, K] and ``out`` the gate's SiLU
    times the up product.  ``out`` bf16 or fp32 [rows, N] (default bf16); rows
    from ``offsets[E]`` on are left as they are.  See
    ``skinny_experts_gemm_bf16``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _on(stream, xs.device):
            return experts_gemm(xs, offsets, w, out, activation)
    rows, K, ldx = _rows(xs, "xs", torch.bfloat16)
    act = _ACTS.get(activation)
    if act is None:
        raise ValueError(f"activation must be 'swiglu' or None, not {activation!r}")
    E, wrows = w.shape[0], w.shape[1]
    if act and wrows % 2:
        raise ValueError(f"swiglu needs gate and up rows, not {wrows} rows")
    N = wrows // 2 if act else wrows
    ldw, ldwe = _stack(w, "w", wrows, K)
    fp = _flat(offsets, "offsets", E + 1, torch.int32)
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=xs.device)
    orows, ocols, ldy = _rows(out, "out")
    if orows != rows or ocols != N:
        raise ValueError(f"out must be {(rows, N)}, not {(orows, ocols)}")
    st = _lib().skinny_experts_gemm_bf16(xs.data_ptr(), ldx, rows, fp, w.data_ptr(), ldw, ldwe, E, N, K, act,
                                         _dtype(out, "out"), out.data_ptr(), ldy, _current(xs.device))
    if st:
        _refused(st, "skinny_experts_gemm_bf16")
    return out


def lora_workspace(M, N, R, out_dtype):
    """Bytes of workspace of :func:`lora_gemm` for an ``out`` of ``out_dtype``."""
    if torch is None:
        _import_torch()
    _fits_int("M, N and R", M, N, R)
    return skinny_lora_workspace(M, N, R, SKINNY_BF16 if out_dtype == torch.bfloat16 else SKINNY_F32)


def lora_gemm(x, w, a, b, adapters, ranks=None, scales=None, out=None, workspace=None, stream=None):
    """A shared projection with a low-rank adapter per token: ``out[m] = x[m] .
    w^T + scales[i] (x[m] . a[i]^T) . b[i]^T`` with ``i = adapters[m]`` (none
    when outside ``[0, L)``), ``x`` bf16 [M, K], ``w`` bf16 [N, K], ``a`` bf16
    [L, R, K], ``b`` bf16 [L, N, R], ``ranks`` int32 [L] (what lies past an
    adapter's rank is not used), ``scales`` fp32 [L], ``out`` fp32 (default)
    or bf16 [M, N].  See ``skinny_lora_gemm_bf16``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _on(stream, x.device):
            return lora_gemm(x, w, a, b, adapters, ranks, scales, out, workspace)
    M, K, ldx = _rows(x, "x", torch.bfloat16)
    N, wcols, ldw = _rows(w, "w", torch.bfloat16)
    L, R = a.shape[0], a.shape[1]
    if wcols != K or b.shape[0] != L:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}, a {tuple(a.shape)}, b {tuple(b.shape)}")
    lda, ldae = _stack(a, "a", R, K)
    ldb, ldbe = _stack(b, "b", N, R)
    ip = _flat(adapters, "adapters", M, torch.int32)
    rp = 0 if ranks is None else _flat(ranks, "ranks", L, torch.int32)
    sp = 0 if scales is None else _flat(scales, "scales", L, torch.float32)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    orows, ocols, ldy = _rows(out, "out")
    ot = _dtype(out, "out")
    if orows != M or ocols != N:
        raise ValueError(f"out must be {(M, N)}, not {(orows, ocols)}")
    if workspace is None:
        workspace = torch.empty(skinny_lora_workspace(M, N, R, ot), dtype=torch.uint8, device=x.device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    st = _lib().skinny_lora_gemm_bf16(x.data_ptr(), ldx, w.data_ptr(), ldw, a.data_ptr(), lda, ldae, b.data_ptr(), ldb,
                                      ldbe, ip, rp, sp, L, R, out.data_ptr(), ldy, M, N, K, ot, workspace.data_ptr(),
                                      workspace.nbytes, _current(x.device))
    if st:
        _refused(st, "skinny_lora_gemm_bf16")
    return out
