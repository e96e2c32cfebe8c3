"""A dense layer's operators around the decode projections: a product with
bias, activation and residual in its epilogue (both projections of a gated
feed-forward block among them), norms of queries and keys for each head with
the position rotation in the same pass, and the backward passes of both.

As in the package itself, the ``skinny_*`` functions carry the C names of
``include/skinny_layer.h`` and only marshal arguments; the tensor functions
(:func:`linear`, :func:`linear_grad`, :func:`qk_norm_rope`,
:func:`qk_norm_rope_grad`) take CUDA tensors, allocate what is not given on
the stream they launch on, and raise on a refusal.
"""
from __future__ import annotations

import ctypes
import struct

import latency_skinny_bf16_gb300 as _sk

from . import experts as _ex

SKINNY_ACT_SILU = 2
SKINNY_ACT_GELU = 3
SKINNY_ACT_GEGLU = 4
SKINNY_MAX_HEAD = 512
SKINNY_MAX_AXES = 8

__all__ = [
    "SKINNY_ACT_SILU", "SKINNY_ACT_GELU", "SKINNY_ACT_GEGLU", "SKINNY_MAX_HEAD", "SKINNY_MAX_AXES",
    "skinny_heads_t", "skinny_rotation_t",
    "skinny_linear_bf16", "skinny_linear_workspace", "skinny_linear_grad_bf16", "skinny_linear_grad_workspace",
    "skinny_qk_norm_rope", "skinny_qk_norm_rope_grad", "skinny_qk_norm_rope_grad_workspace",
    "linear", "linear_workspace", "linear_grad", "linear_grad_workspace",
    "qk_norm_rope", "qk_norm_rope_grad", "qk_norm_rope_grad_workspace",
]

SYMBOLS = ("skinny_linear_bf16", "skinny_linear_workspace", "skinny_linear_grad_bf16", "skinny_linear_grad_workspace",
           "skinny_qk_norm_rope", "skinny_qk_norm_rope_grad", "skinny_qk_norm_rope_grad_workspace")

_ACTS = {None: _ex.SKINNY_ACT_NONE, "none": _ex.SKINNY_ACT_NONE, "silu": SKINNY_ACT_SILU, "gelu": SKINNY_ACT_GELU,
         "swiglu": _ex.SKINNY_ACT_SWIGLU, "geglu": SKINNY_ACT_GEGLU}
_GATED = (_ex.SKINNY_ACT_SWIGLU, SKINNY_ACT_GEGLU)
_fits_int = _sk._fits_int
_lib = _ex._lib
_rows = _ex._rows
_refused = _ex._refused


class skinny_heads_t(ctypes.Structure):
    """Heads of queries or keys, as in the header."""
    _fields_ = [("x", ctypes.c_void_p), ("st", ctypes.c_int64), ("sh", ctypes.c_int64), ("w", ctypes.c_void_p),
                ("H", ctypes.c_int)]


class skinny_rotation_t(ctypes.Structure):
    """How heads are turned, as in the header."""
    _fields_ = [("table", ctypes.c_void_p), ("P", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("pair_axis", ctypes.c_void_p), ("axes", ctypes.c_int), ("R", ctypes.c_int), ("interleaved", ctypes.c_int)]


# The same bytes, without a field's conversions: 0.2 us, and 0.5 to 0.8 as a structure.
_pack_heads = struct.Struct("PqqPi4x").pack
_pack_rotation = struct.Struct("PqPPiii4x").pack
_NO_HEADS = _pack_heads(0, 0, 0, 0, 0)
_NO_TURN = _pack_rotation(0, 1, 0, 0, 1, 0, 0)
_rope = _rope_grad = None       # the entry points of the tensor functions, by bytes


def bind(lib: ctypes.CDLL) -> None:
    global _rope, _rope_grad
    vp, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    hp, rp = ctypes.POINTER(skinny_heads_t), ctypes.POINTER(skinny_rotation_t)
    lib.skinny_linear_bf16.argtypes = [vp, i, vp, i, vp, vp, i, vp, i, vp, i, i, i, i, i, i, vp, ll, vp]
    lib.skinny_linear_workspace.argtypes = [vp, i, vp, i, i, i, i, i]
    lib.skinny_linear_grad_bf16.argtypes = [vp, i, vp, i, vp, i, vp, i, vp, i, vp, i, vp, i, i, i, i, vp, ll, vp]
    lib.skinny_linear_grad_workspace.argtypes = [vp, i, vp, i, vp, i, i, i, i, i]
    lib.skinny_qk_norm_rope.argtypes = [hp, hp, rp, i, i, i, f, i, vp, ll, ll, vp, ll, ll, vp]
    lib.skinny_qk_norm_rope_grad.argtypes = [vp, ll, ll, vp, ll, ll, hp, hp, rp, i, i, i, f, i, vp, ll, ll, vp, ll, ll, vp,
                                             vp, vp, ll, vp]
    lib.skinny_qk_norm_rope_grad_workspace.argtypes = [i, i, i, i]
    for name in SYMBOLS:
        getattr(lib, name).restype = ll if name.endswith("workspace") else i
    _rope, _rope_grad = lib["skinny_qk_norm_rope"], lib["skinny_qk_norm_rope_grad"]
    for f, named in ((_rope, lib.skinny_qk_norm_rope), (_rope_grad, lib.skinny_qk_norm_rope_grad)):
        f.argtypes = [vp if a in (hp, rp) else a for a in named.argtypes]
        f.restype = i


# ---------------------------------------------------------------- C-named wrappers (raw pointers)

def skinny_linear_bf16(X: int, ldx: int, W: int, ldw: int, bias: int, R: int, ldr: int, Y: int, ldy: int, Z: int,
                       ldz: int, M: int, N: int, K: int, act: int, out_dtype: int, workspace: int,
                       workspace_bytes: int, stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_linear_bf16(X, ldx, W, ldw, bias, R, ldr, Y, ldy, Z, ldz, M, N, K, act, out_dtype, workspace,
                                     workspace_bytes, stream)


def skinny_linear_workspace(X: int, ldx: int, W: int, ldw: int, M: int, N: int, K: int, act: int) -> int:
    """Bytes of workspace of skinny_linear_bf16; 0 for sizes it refuses."""
    return _lib().skinny_linear_workspace(X, ldx, W, ldw, M, N, K, act)


def skinny_linear_grad_bf16(dY: int, lddy: int, X: int, ldx: int, W: int, ldw: int, Z: int, ldz: int, dX: int,
                            lddx: int, dW: int, lddw: int, dbias: int, M: int, N: int, K: int, act: int,
                            workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_linear_grad_bf16(dY, lddy, X, ldx, W, ldw, Z, ldz, dX, lddx, dW, lddw, dbias, M, N, K, act,
                                          workspace, workspace_bytes, stream)


def skinny_linear_grad_workspace(dY: int, lddy: int, X: int, ldx: int, W: int, ldw: int, M: int, N: int, K: int,
                                 act: int) -> int:
    """Bytes of workspace of skinny_linear_grad_bf16; 0 for sizes it refuses."""
    return _lib().skinny_linear_grad_workspace(dY, lddy, X, ldx, W, ldw, M, N, K, act)


def skinny_qk_norm_rope(q: skinny_heads_t, k: skinny_heads_t, rot: skinny_rotation_t, T: int, D: int, norm: int,
                        eps: float, dtype: int, q_out: int, q_st: int, q_sh: int, k_out: int, k_st: int, k_sh: int,
                        stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_qk_norm_rope(q, k, rot, T, D, norm, eps, dtype, q_out, q_st, q_sh, k_out, k_st, k_sh, stream)


def skinny_qk_norm_rope_grad(dq: int, dq_st: int, dq_sh: int, dk: int, dk_st: int, dk_sh: int, q: skinny_heads_t,
                             k: skinny_heads_t, rot: skinny_rotation_t, T: int, D: int, norm: int, eps: float,
                             dtype: int, q_grad: int, qg_st: int, qg_sh: int, k_grad: int, kg_st: int, kg_sh: int,
                             q_wgrad: int, k_wgrad: int, workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    """Raw C call; returns the skinny_status_t."""
    return _lib().skinny_qk_norm_rope_grad(dq, dq_st, dq_sh, dk, dk_st, dk_sh, q, k, rot, T, D, norm, eps, dtype, q_grad,
                                           qg_st, qg_sh, k_grad, kg_st, kg_sh, q_wgrad, k_wgrad, workspace,
                                           workspace_bytes, stream)


def skinny_qk_norm_rope_grad_workspace(T: int, q_heads: int, k_heads: int, D: int) -> int:
    """Bytes of workspace of skinny_qk_norm_rope_grad; 0 for sizes it refuses."""
    return _lib().skinny_qk_norm_rope_grad_workspace(T, q_heads, k_heads, D)


# ---------------------------------------------------------------- tensors

torch = None    # imported by the first call that takes tensors: the C-named functions need none


def _import_torch():
    global torch, _bf16, _f32, _i32, _device
    if _ex.torch is None:
        _ex._import_torch()
    torch = _ex.torch
    _bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here(t, name):
    """The current device, on which the library launches and every tensor has to be."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, not on {t.device}")
    at = _device()
    if t.get_device() != at:
        raise ValueError(f"{name} is on {t.device}, and the current device is cuda:{at}")
    return at


def _elsewhere(t, name, at):
    raise ValueError(f"{name} is on {t.device}, and the other tensors on cuda:{at}")


def _act(activation, wrows):
    """(act, N) of a weight of `wrows` rows."""
    act = _ACTS.get(activation)
    if act is None:
        raise ValueError(f"activation must be None, 'silu', 'gelu', 'swiglu' or 'geglu', not {activation!r}")
    if act in _GATED:
        if wrows % 2:
            raise ValueError(f"{activation} needs gate and up rows, not {wrows} rows")
        return act, wrows // 2
    return act, wrows


def _matrix(t, name, rows, cols, dtype, at):
    """(address, row stride) of a CUDA matrix of that size; None: (0, 0)."""
    if t is None:
        return 0, 0
    if t.get_device() != at:
        _elsewhere(t, name, at)
    m, n, ld = _rows(t, name, dtype)
    if m != rows or n != cols:
        raise ValueError(f"{name} must be {(rows, cols)}, not {(m, n)}")
    return t.data_ptr(), ld


def _vector(t, name, n, dtype, at):
    """Address of a contiguous CUDA tensor of n elements; None: 0."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != at:
        _elsewhere(t, name, at)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} elements")
    return t.data_ptr()


def _space(workspace, at):
    """(address, bytes) of a workspace."""
    if workspace.get_device() != at or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{at}")
    return workspace.data_ptr(), workspace.nbytes


def linear_workspace(x, w, activation=None):
    """Bytes of workspace of :func:`linear` for these tensors (0 for most)."""
    if torch is None:
        _import_torch()
    M, K, ldx = _rows(x, "x", torch.bfloat16)
    wrows, _, ldw = _rows(w, "w", torch.bfloat16)
    act, N = _act(activation, wrows)
    return _lib().skinny_linear_workspace(x.data_ptr(), ldx, w.data_ptr(), ldw, M, N, K, act)


def linear(x, w, bias=None, activation=None, residual=None, out=None, pre=None, workspace=None, stream=None):
    """``z = x . w^T + bias``, and ``out = act(z) + residual`` (``activation``
    None, "silu" or "gelu", the tanh form), or, with "swiglu" and "geglu" and
    ``w`` [2N, K], ``out = act(z[:, :N]) * z[:, N:] + residual``: ``x`` bf16
    [M, K], ``bias`` bf16, ``out`` bf16 (default) or fp32 [M, N], ``residual``
    as ``out`` (it may be ``out`` itself).  ``pre``, bf16 and as wide as ``w``
    has rows, keeps z for :func:`linear_grad`.  Any number of rows.  Rows that
    do not lie on 16-byte boundaries are laid out in ``workspace`` on every
    call (:func:`linear_workspace` bytes, allocated where none is given).  See
    ``skinny_linear_bf16``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _ex._on(stream, x.device):
            return linear(x, w, bias, activation, residual, out, pre, workspace)
    at = _here(x, "x")
    M, K, ldx = _rows(x, "x", _bf16)
    wrows, wcols, ldw = _rows(w, "w", _bf16)
    if wcols != K:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}")
    if w.get_device() != at:
        _elsewhere(w, "w", at)
    act, N = _act(activation, wrows)
    if out is None:
        out = torch.empty((M, N), dtype=_bf16 if residual is None else residual.dtype, device=x.device)
    yp, ldy = _matrix(out, "out", M, N, None, at)
    rp, ldr = _matrix(residual, "residual", M, N, out.dtype, at)
    zp, ldz = _matrix(pre, "pre", M, wrows, _bf16, at)
    bp = _vector(bias, "bias", wrows, _bf16, at)
    ot = _ex._dtype(out, "out")
    xp, wp = x.data_ptr(), w.data_ptr()
    lib = _lib()
    sp = sb = 0
    if workspace is None:
        if (xp | wp) & 15 or (ldx | ldw) & 7:        # else none is needed
            workspace = torch.empty(lib.skinny_linear_workspace(xp, ldx, wp, ldw, M, N, K, act), dtype=torch.uint8,
                                    device=x.device)
    if workspace is not None:
        sp, sb = _space(workspace, at)
    st = lib.skinny_linear_bf16(xp, ldx, wp, ldw, bp, rp, ldr, yp, ldy, zp, ldz, M, N, K, act, ot, sp, sb,
                                _ex._current(x.device))
    if st:
        _refused(st, "skinny_linear_bf16")
    return out


def linear_grad_workspace(dy, x, w, activation=None):
    """Bytes of workspace of :func:`linear_grad` for these tensors."""
    if torch is None:
        _import_torch()
    _, _, lddy = _rows(dy, "dy", torch.bfloat16)
    M, K, ldx = _rows(x, "x", torch.bfloat16)
    wrows, _, ldw = _rows(w, "w", torch.bfloat16)
    act, N = _act(activation, wrows)
    return _lib().skinny_linear_grad_workspace(dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), ldw, M, N, K, act)


def linear_grad(dy, x, w, pre=None, activation=None, dx=None, dw=None, dbias=None, input_grad=True, weight_grad=True,
                bias_grad=False, workspace=None, stream=None):
    """The gradients of :func:`linear` for ``dy`` bf16 [M, N]: returns ``(dx,
    dw, dbias)``, bf16 as ``x`` and ``w`` and fp32 [rows of ``w``], None where
    ``input_grad``, ``weight_grad`` or ``bias_grad`` leaves one out.  ``pre``
    is what the forward pass kept (not used without an activation); the
    residual's gradient is ``dy``.  See ``skinny_linear_grad_bf16``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _ex._on(stream, dy.device):
            return linear_grad(dy, x, w, pre, activation, dx, dw, dbias, input_grad, weight_grad, bias_grad, workspace)
    at = _here(dy, "dy")
    M, K, ldx = _rows(x, "x", _bf16)
    wrows, wcols, ldw = _rows(w, "w", _bf16)
    if wcols != K:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}")
    for t, name in ((x, "x"), (w, "w")):
        if t.get_device() != at:
            _elsewhere(t, name, at)
    act, N = _act(activation, wrows)
    yp, lddy = _matrix(dy, "dy", M, N, _bf16, at)
    if act and pre is None:
        raise ValueError(f"{activation} needs pre, what the forward pass kept")
    zp, ldz = _matrix(pre, "pre", M, wrows, _bf16, at) if act else (0, 0)
    for wanted, t, name in ((input_grad, dx, "dx"), (weight_grad, dw, "dw"), (bias_grad, dbias, "dbias")):
        if not wanted and t is not None:
            raise ValueError(f"{name} is given, and not asked for")
    if input_grad and dx is None:
        dx = torch.empty((M, K), dtype=_bf16, device=dy.device)
    if weight_grad and dw is None:
        dw = torch.empty((wrows, K), dtype=_bf16, device=dy.device)
    if bias_grad and dbias is None:
        dbias = torch.empty(wrows, dtype=_f32, device=dy.device)
    gxp, lddx = _matrix(dx, "dx", M, K, _bf16, at)
    gwp, lddw = _matrix(dw, "dw", wrows, K, _bf16, at)
    gbp = _vector(dbias, "dbias", wrows, _f32, at)
    xp, wp = x.data_ptr(), w.data_ptr()
    lib = _lib()
    if workspace is None:
        workspace = torch.empty(lib.skinny_linear_grad_workspace(yp, lddy, xp, ldx, wp, ldw, M, N, K, act),
                                dtype=torch.uint8, device=dy.device)
    sp, sb = _space(workspace, at)
    st = lib.skinny_linear_grad_bf16(yp, lddy, xp, ldx, wp, ldw, zp, ldz, gxp, lddx, gwp, lddw, gbp, M, N, K, act, sp, sb,
                                     _ex._current(dy.device))
    if st:
        _refused(st, "skinny_linear_grad_bf16")
    return dx, dw, dbias


def _view(t, name, at, shape=None, dtype=None):
    """(address, token stride, head stride) of CUDA heads [T, H, D] with unit stride along D."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if shape is not None and (t.shape != shape or t.dtype is not dtype):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    if t.get_device() != at:
        _elsewhere(t, name, at)
    st, sh, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} needs unit stride along its last dimension")
    return t.data_ptr(), st, sh


def _heads(q, k, q_weight, k_weight, table, positions, eps, pair_axis, interleaved):
    """The header's structures for these tensors, and (T, D, dtype, device)."""
    at = _here(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, D], not {tuple(q.shape)}")
    T, Hq, D = q.shape
    dtype = q.dtype
    dt = _ex._dtype(q, "q")
    if eps is None and (q_weight is not None or k_weight is not None):
        raise ValueError("weights are given, and no eps: without eps there is no norm")
    if (T | Hq | D) >> 31:
        _fits_int("q", T, Hq, D)
    p, st, sh = _view(q, "q", at)
    hq = _pack_heads(p, st, sh, _vector(q_weight, "q_weight", D, dtype, at), Hq)
    if k is None:
        if k_weight is not None:
            raise ValueError("k_weight is given, and no k")
        hk = _NO_HEADS
    else:
        if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or k.dtype is not dtype:
            raise ValueError(f"shape mismatch: q {dtype} {tuple(q.shape)}, k {k.dtype} {tuple(k.shape)}")
        p, st, sh = _view(k, "k", at)
        Hk = k.shape[1]
        if Hk >> 31:
            _fits_int("k", Hk)
        hk = _pack_heads(p, st, sh, _vector(k_weight, "k_weight", D, dtype, at), Hk)
    if table is None:
        rot = _NO_TURN
    else:
        if table.dim() != 2 or positions is None:
            raise ValueError("a table [positions, R] goes with the tokens' positions")
        P, R = table.shape
        d = positions.dim()
        axes = 1 if d == 1 else positions.shape[0]
        if d != 1 and d != 2:
            raise ValueError(f"positions must be [tokens] or [axes, tokens], not {tuple(positions.shape)}")
        if (R | axes) >> 31:
            _fits_int("table", R, axes)
        rot = _pack_rotation(_vector(table, "table", P * R, _f32, at), P,
                             _vector(positions, "positions", axes * T, _i32, at),
                             _vector(pair_axis, "pair_axis", R // 2, _i32, at), axes, R, 1 if interleaved else 0)
    return hq, hk, rot, T, D, dt, at


def qk_norm_rope(q, k, q_weight=None, k_weight=None, table=None, positions=None, eps=1e-6, pair_axis=None,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """Each head of ``q`` [T, Hq, D] and ``k`` [T, Hk, D] (bf16 or fp32, views
    into a projection's rows are taken as they are; ``k`` may be None)
    normalised, ``x / sqrt(mean(x^2) + eps) * weight`` (``eps=None``: no norm;
    a weight of None: ones), and turned by its token's position: ``table`` fp32
    [P, R] holds the cosines of the R / 2 pairs, then their sines;
    ``positions`` int32 [T], or [axes, T] with ``pair_axis`` int32 [R / 2], the
    axis that turns each pair.  Pairs are halves, (i, R/2 + i), or neighbours
    when ``interleaved``; elements from R on are not turned, nor is a token
    whose position is outside the table.  Returns ``(q_out, k_out)``, which may
    be the inputs themselves.  See ``skinny_qk_norm_rope``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _ex._on(stream, q.device):
            return qk_norm_rope(q, k, q_weight, k_weight, table, positions, eps, pair_axis, interleaved, q_out, k_out)
    hq, hk, rot, T, D, dt, at = _heads(q, k, q_weight, k_weight, table, positions, eps, pair_axis, interleaved)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    qp, qst, qsh = _view(q_out, "q_out", at, q.shape, q.dtype)
    kp = kst = ksh = 0
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        kp, kst, ksh = _view(k_out, "k_out", at, k.shape, k.dtype)
    elif k_out is not None:
        raise ValueError("k_out is given, and no k")
    if _rope is None:
        _lib()
    st = _rope(hq, hk, rot, T, D, eps is not None, eps or 0.0, dt, qp, qst, qsh, kp, kst, ksh, _ex._current(q.device))
    if st:
        _refused(st, "skinny_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_grad_workspace(T, q_heads, k_heads, D):
    """Bytes of workspace of :func:`qk_norm_rope_grad`."""
    _fits_int("T, heads and D", T, q_heads, k_heads, D)
    return skinny_qk_norm_rope_grad_workspace(T, q_heads, k_heads, D)


def qk_norm_rope_grad(dq, dk, q, k, q_weight=None, k_weight=None, table=None, positions=None, eps=1e-6, pair_axis=None,
                      interleaved=False, dq_in=None, dk_in=None, dq_weight=None, dk_weight=None, weight_grad=True,
                      workspace=None, stream=None):
    """The gradients of :func:`qk_norm_rope` for ``dq`` and ``dk``: returns
    ``(dq_in, dk_in, dq_weight, dk_weight)``, the weights' in fp32 [D] (None
    without a norm, or with ``weight_grad=False``; a weight of None counts as
    ones, and its gradient is given).  ``dq_in`` may be ``dq`` itself.  See
    ``skinny_qk_norm_rope_grad``."""
    if torch is None:
        _import_torch()
    if stream is not None:
        with _ex._on(stream, q.device):
            return qk_norm_rope_grad(dq, dk, q, k, q_weight, k_weight, table, positions, eps, pair_axis, interleaved,
                                     dq_in, dk_in, dq_weight, dk_weight, weight_grad, workspace)
    hq, hk, rot, T, D, dt, at = _heads(q, k, q_weight, k_weight, table, positions, eps, pair_axis, interleaved)
    dqp, dqst, dqsh = _view(dq, "dq", at, q.shape, q.dtype)
    if dq_in is None:
        dq_in = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    qp, qst, qsh = _view(dq_in, "dq_in", at, q.shape, q.dtype)
    dkp = dkst = dksh = kp = kst = ksh = 0
    if k is not None:
        dkp, dkst, dksh = _view(dk, "dk", at, k.shape, k.dtype)
        if dk_in is None:
            dk_in = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        kp, kst, ksh = _view(dk_in, "dk_in", at, k.shape, k.dtype)
    elif dk is not None or dk_in is not None or dk_weight is not None:
        raise ValueError("gradients of keys are given, and no k")
    wqp = wkp = sp = sb = 0
    norm = eps is not None
    if norm and weight_grad:
        if dq_weight is None:
            dq_weight = torch.empty(D, dtype=_f32, device=q.device)
        wqp = _vector(dq_weight, "dq_weight", D, _f32, at)
        if k is not None:
            if dk_weight is None:
                dk_weight = torch.empty(D, dtype=_f32, device=q.device)
            wkp = _vector(dk_weight, "dk_weight", D, _f32, at)
        if workspace is None:
            need = skinny_qk_norm_rope_grad_workspace(T, q.shape[1], 0 if k is None else k.shape[1], D)
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        sp, sb = _space(workspace, at)
    elif dq_weight is not None or dk_weight is not None:
        raise ValueError("a weight's gradient is given, and not asked for")
    if _rope_grad is None:
        _lib()
    st = _rope_grad(dqp, dqst, dqsh, dkp, dkst, dksh, hq, hk, rot, T, D, norm, eps or 0.0, dt, qp, qst, qsh, kp, kst, ksh,
                    wqp, wkp, sp, sb, _ex._current(q.device))
    if st:
        _refused(st, "skinny_qk_norm_rope_grad")
    return dq_in, dk_in, dq_weight, dk_weight
