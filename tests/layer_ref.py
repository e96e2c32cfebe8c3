"""Plain forms, in 64 bits on the CPU, of a dense layer's operators, and the
bounds that their results are held to."""
import math

import torch

GATED = ("swiglu", "geglu")
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float64: 0.0}    # half a step of a rounding


def act_both(act, z):
    """(act(z), act'(z)) in 64 bits."""
    if act in (None, "none"):
        return z, torch.ones_like(z)
    c = math.sqrt(2 / math.pi)
    u, du = (z, torch.ones_like(z)) if act in ("silu", "swiglu") else \
        (2 * c * (z + 0.044715 * z ** 3), 2 * c * (1 + 3 * 0.044715 * z ** 2))
    s = torch.sigmoid(u)
    return z * s, s + z * s * (1 - s) * du


def linear(x, w, bias, act, residual):
    """(y, z, the sum of the products' absolute values with the bias' [M, rows])."""
    x, w = x.double().cpu(), w.double().cpu()
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias.double().cpu(), size + bias.double().cpu().abs()
    N = w.shape[0] // 2 if act in GATED else w.shape[0]
    y = act_both(act, z[:, :N])[0]
    if act in GATED:
        y = y * z[:, N:]
    if residual is not None:
        y = y + residual.double().cpu()
    return y, z, size


def linear_bound(y, z, size, act, residual, dtype):
    """How far an output may be off.  A sum z comes within dz = 1e-5 of its
    terms' sum (tensor-core chains of 16 MMAs and rounded adds, as the plain
    products).  SiLU and GELU have slopes within 1.13, and beyond the sum's
    error are computed in fp32 with an exponential (error 2 units of |u| + 1
    steps: exp(u) turns an error of 2^-24 |u| of its argument into one of that
    size relative to it), a division and a product: 2^-20 of the value and of
    the products beside it covers all of it while |u| stays below 88, past
    which the factor is 0 or 1.  Then the output's one rounding."""
    N = y.shape[1]
    dz = 1e-5 * size + 1e-6
    err = 1.2 * dz[:, :N]
    if act in GATED:
        a = act_both(act, z[:, :N])[0].abs()
        err = err * (z[:, N:].abs() + dz[:, N:]) + a * dz[:, N:]
    own = (y if residual is None else y - residual.double().cpu()).abs()
    err = err + 2.0 ** -19 * own + (0 if act in (None, "none") else 2.0 ** -20 * dz[:, :N])
    if residual is not None:
        err = err + 2.0 ** -23 * (own + residual.double().cpu().abs())
    return err + STEP[dtype] * 1.01 * (y.abs() + err) + 1e-30


def linear_dz(dy, z, act):
    """dZ [M, rows] in 64 bits from dY and the kept Z."""
    dy = dy.double().cpu()
    if act in (None, "none"):
        return dy
    z = z.double().cpu()
    if act in GATED:
        N = dy.shape[1]
        a, da = act_both(act, z[:, :N])
        return torch.cat([dy * z[:, N:] * da, dy * a], dim=1)
    return dy * act_both(act, z)[1]


def linear_grad(dy, x, w, z, act):
    """(dx, dw, dbias) and their bounds.  dZ is off by a few fp32 steps (2^-19,
    as above; act' may cancel, which the 2^-19 of max(|z|, 1) |dy| covers) and,
    with an activation, by a rounding to bf16; the sums by 1e-5 of their terms;
    the results by a rounding to bf16.  dbias sums what was not rounded, up to
    M terms in fp32 by chains of at most M / 64 + 16 adds."""
    dz = linear_dz(dy, z, act)
    x, w, d64 = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    if act in (None, "none"):
        edz = torch.zeros_like(dz)
        fine = edz
    else:
        zz = z.double().cpu()
        N = d64.shape[1]
        big = d64.abs() * zz[:, :N].abs().clamp(min=1)
        if act in GATED:
            big = torch.cat([big * zz[:, N:].abs(), big], dim=1)
        fine = 2.0 ** -19 * big
        edz = fine + 2.0 ** -8 * (dz.abs() + fine)
    M = dy.shape[0]
    out = []
    for a, b, ea in ((dz, w, edz), (dz.t(), x, edz.t())):
        v = a @ b
        err = ea @ b.abs() + 1e-5 * ((a.abs() + ea) @ b.abs()) + 1e-30
        out.append((v, err + 2.0 ** -8 * 1.01 * (v.abs() + err)))
    s = dz.sum(0)
    out.append((s, fine.sum(0) + (M / 64 + 80) * 2.0 ** -24 * (dz.abs() + fine).sum(0) + 1e-30))
    return out


# ------------------------------------------------------------------ heads

def angles(table, positions, pair_axis, T):
    """(cos, sin) [T, R / 2] in 64 bits; a position or an axis outside does not turn."""
    table = table.double().cpu()
    P, R = table.shape
    half = R // 2
    positions = positions.cpu().reshape(-1, T).long()
    axis = torch.zeros(half, dtype=torch.long) if pair_axis is None else pair_axis.cpu().long()
    inside = (axis >= 0) & (axis < positions.shape[0])
    at = positions[axis.clamp(0, positions.shape[0] - 1)].t()               # [T, pairs]
    ok = inside[None] & (at >= 0) & (at < P)
    at = at.clamp(0, P - 1)
    pair = torch.arange(half)[None]
    one, zero = torch.ones((), dtype=torch.double), torch.zeros((), dtype=torch.double)
    return torch.where(ok, table[at, pair], one), torch.where(ok, table[at, half + pair], zero)


def pairs(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, R // 2 + i)


def turned(x, cos, sin, interleaved, back=False):
    y = x.clone()
    a, b = pairs(2 * cos.shape[1], interleaved)
    c, s = cos[:, None], (-sin if back else sin)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def heads(x, w, cos, sin, eps, interleaved, dtype):
    """(y, bound): the sum of squares, the root, the division and two products
    are 2^-19 relative for a head of 512 (its sum: 512 / 32 + 5 + 8 adds), the
    rotation's products and sum 3 * 2^-24 of both terms."""
    x = x.double().cpu()
    n = x
    if eps is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            n = n * w.double().cpu()
    if cos is None:
        y, size = n, n.abs()
    else:
        y, size = turned(n, cos, sin, interleaved), turned(n.abs(), cos.abs(), -sin.abs(), interleaved)
        a, b = pairs(2 * cos.shape[1], interleaved)
        size[..., b] = n.abs()[..., b] * cos.abs()[:, None] + n.abs()[..., a] * sin.abs()[:, None]
    err = 2.0 ** -18 * size
    return y, err + STEP[dtype] * 1.01 * (y.abs() + err) + 1e-30


def heads_grad(dy, x, w, cos, sin, eps, interleaved, dtype):
    """((dx, bound), (dw, bound)): as above; dx is a difference of two terms,
    each within 2^-18 of the sums of their own absolute values.  dw sums
    T * H terms, at most T * H / 8 + 600 in a chain."""
    d = dy.double().cpu()
    g, size = d, d.abs()
    if cos is not None:
        g = turned(d, cos, sin, interleaved, back=True)
        a, b = pairs(2 * cos.shape[1], interleaved)
        size = d.abs().clone()
        size[..., a] = d.abs()[..., a] * cos.abs()[:, None] + d.abs()[..., b] * sin.abs()[:, None]
        size[..., b] = d.abs()[..., b] * cos.abs()[:, None] + d.abs()[..., a] * sin.abs()[:, None]
    if eps is None:
        err = 2.0 ** -18 * size
        return (g, err + STEP[dtype] * 1.01 * (g.abs() + err) + 1e-30), None
    x = x.double().cpu()
    w64 = torch.ones(x.shape[-1], dtype=torch.double) if w is None else w.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h, hs = g * w64, size * w64.abs()
    dx = r * h - x * r ** 3 * (h * x).mean(-1, keepdim=True)
    err = 2.0 ** -17 * (r * hs + x.abs() * r ** 3 * (hs * x.abs()).mean(-1, keepdim=True))
    terms = g * x * r
    dw = terms.sum((0, 1))
    n = x.shape[0] * x.shape[1]
    dwe = (2.0 ** -18 + (n / 8 + 600) * 2.0 ** -24) * (size * x.abs() * r).sum((0, 1)) + 1e-30
    return (dx, err + STEP[dtype] * 1.01 * (dx.abs() + err) + 1e-30), (dw, dwe)


def check(got, want, bound, what=""):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - want).abs() / bound)[bad].max():.3g} "
                           f"of the bound, first at {bad.nonzero()[0].tolist()}")
