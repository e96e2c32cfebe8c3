"""Inputs and outputs as columns of one buffer side by side, as apart."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk

pytestmark = pytest.mark.gpu

KERNELS = {"any": 0, "pair": sk.SKINNY_BACKEND_TCGEN05, "split": sk.SKINNY_BACKEND_SPLITK}


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("pdl", [0, 1])
@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (40, 72, 136), (33, 61, 127), (700, 264, 320), (300, 7, 9)])
def test_side_by_side(M, N, K, pdl, act, kernel):
    g = torch.Generator(device="cuda").manual_seed(M)
    rows = 2 * N if act == "swiglu" else N

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    w, bias = rand(rows, K), rand(rows)
    # [x | out | pre | residual | dy | dx] of a token, and [w | dw] of an output
    widths = [K, N, rows, N, N, K]
    buf = rand(M, sum(widths) + 5)
    both = torch.cat([w, rand(rows, K)], dim=1)
    x, out, pre, res, dy, dx = buf[:, :sum(widths)].split(widths, dim=1)
    w1, dw1 = both.split(K, dim=1)
    apart = [t.contiguous().clone() for t in (x, res, dy)]
    z = torch.empty((M, rows), dtype=torch.bfloat16, device="cuda")
    kw = dict(activation=act)
    with sk.options(pdl=pdl, backend=KERNELS[kernel]):
        want = sk.linear(apart[0], w, bias=bias, residual=apart[1], pre=z, **kw)
        dwant = sk.linear_grad(apart[2], apart[0], w, pre=z if act else None, bias_grad=True, **kw)
        sk.linear(x, w1, bias=bias, residual=res, out=out, pre=pre, **kw)
        got = sk.linear_grad(dy, x, w1, pre=pre if act else None, dx=dx, dw=dw1, bias_grad=True, **kw)
    assert torch.equal(out, want) and torch.equal(pre, z)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], dwant[:2]))
    # the bias gradient's order of adds goes by the rows' boundaries
    size = dwant[2].abs() + M * 8.0
    assert ((got[2] - dwant[2]).abs() <= 2.0 ** -20 * size).all()
    assert torch.equal(x, apart[0]) and torch.equal(res, apart[1]) and torch.equal(dy, apart[2]) and torch.equal(w1, w)
    assert sk.skinny_get_device_status() == 0
