"""Plain 64-bit forms of the operators of include/skinny_experts.h, and the
inputs their tests share.  numpy only, one entry at a time where that is the
definition."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                        # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "fp32": U32}  # half a step of the stored types
TINY = {"bf16": 2.0 ** -134, "fp32": 2.0 ** -150}   # half a step below the normal range


def routing(T, k, E, seed, drop=0.0, skew=0.0):
    """ids int32 [T, k] (k different experts a token; -1 where dropped) and fp32 weights."""
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32) if T else np.zeros((0, k), np.int32)
    w = rng.random((T, k)).astype(np.float32)
    if drop:
        ids[rng.random((T, k)) < drop] = -1
        if T > 1:
            ids[T // 2] = -1
    return np.ascontiguousarray(ids), w


def dispatch(ids, E):
    """(pos [T, k], order [T*k], offsets [E+1])."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    live = [f for f in range(T * k) if 0 <= flat[f] < E]
    live.sort(key=lambda f: int(flat[f]))          # stable
    pos = np.full(T * k, -1, np.int32)
    order = np.full(T * k, -1, np.int32)
    for p, f in enumerate(live):
        pos[f] = p
        order[p] = f
    counts = np.bincount(flat[live], minlength=E) if live else np.zeros(E, np.int64)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return pos.reshape(T, k), order, offsets


def combine(ys, pos, w):
    """(y, sum of the magnitudes added) in fp64; w None: ones."""
    T, k = pos.shape
    y = np.zeros((T, ys.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < ys.shape[0]:
                r = ys[pos[t, j]].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
                y[t] += r
                mag[t] += np.abs(r)
    return y, mag


def combine_grad(dy, ys, pos, w):
    """(dys with NaN where no entry names the row, dw, sum of the magnitudes in dw)."""
    T, k = pos.shape
    dys = np.full(ys.shape, np.nan)
    dw = np.zeros((T, k))
    mag = np.zeros((T, k))
    for t in range(T):
        g = dy[t].astype(np.float64)
        for j in range(k):
            p = pos[t, j]
            if 0 <= p < ys.shape[0]:
                dys[p] = g * (1.0 if w is None else float(w[t, j]))
                dw[t, j] = g @ ys[p].astype(np.float64)
                mag[t, j] = np.abs(g) @ np.abs(ys[p].astype(np.float64))
    return dys, dw, mag


def rounded(ref, err, out):
    """How far a value computed within `err` of `ref` and rounded once to `out` may be from ref."""
    return err + HALF[out] * (np.abs(ref) + err) + TINY[out]


def silu_mul(g, u):
    return g / (1.0 + np.exp(-g)) * u


def experts(xs, offsets, w, swiglu):
    """(y, bound on the error of an fp32 evaluation): every sum of products within 1e-5 of the
    sum of their magnitudes, SiLU's slope below 1.1, its evaluation within 8 roundings."""
    rows, K = xs.shape
    N = w.shape[1] // 2 if swiglu else w.shape[1]
    y, err = np.full((rows, N), np.nan), np.zeros((rows, N))
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        h = xs[a:b] @ w[e].T
        mag = 1e-5 * (np.abs(xs[a:b]) @ np.abs(w[e]).T)
        if swiglu:
            g, u, dg, du = h[:, :N], h[:, N:], mag[:, :N], mag[:, N:]
            y[a:b] = silu_mul(g, u)
            s = np.abs(g / (1.0 + np.exp(-g)))
            err[a:b] = 1.1 * dg * np.abs(u) + (s + 1.1 * dg) * du + 8 * U32 * np.abs(y[a:b])
        else:
            y[a:b], err[a:b] = h, mag
    return y, err


def lora(x, w, a, b, adapters, ranks, scales):
    """(y, bound on the error of an fp32 evaluation)."""
    M, K = x.shape
    L, R = a.shape[0], a.shape[1]
    y = x @ w.T
    err = 1e-5 * (np.abs(x) @ np.abs(w).T)
    for m in range(M):
        i = int(adapters[m])
        if not 0 <= i < L:
            continue
        r = R if ranks is None else max(0, min(R, int(ranks[i])))
        s = 1.0 if scales is None else float(scales[i])
        v = s * (a[i, :r] @ x[m])
        dv = abs(s) * (8 + K / 256 + 16) * U32 * (np.abs(a[i, :r]) @ np.abs(x[m]))
        y[m] += b[i, :, :r] @ v
        # the products of a row in eight at a time, then across the lanes, then the base
        err[m] += np.abs(b[i, :, :r]) @ dv + 48 * U32 * (np.abs(b[i, :, :r]) @ np.abs(v)) + U32 * np.abs(y[m])
    return y, 1.01 * err
