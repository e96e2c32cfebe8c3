"""Sums over long depths, nothing of which cancels, against 64 bits.

The header's bound: 1e-5 of the terms' absolute sum up to 32768 steps, 2^-32 of
it more for each step beyond.  It follows from the kernels' adds.  A chain of n
MMAs is off by n 2 2^-24 at most, each add to the long sum by 2^-24:
  split  16 MMAs (1.9e-6), an add for 256 steps:  128 2^-24 at 32768, 9.5e-6 together
  pair   64 MMAs (7.6e-6), an add for 1024 steps:  32 2^-24 at 32768, 9.5e-6 together
  dbias  an add for 512 tokens, 72 beside them:   136 2^-24 at 32768, 8.1e-6
and beyond that an add for 256 steps at most: 2^-24 / 256 = 2^-32 a step."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk

pytestmark = pytest.mark.gpu

KERNELS = {"any": 0, "pair": sk.SKINNY_BACKEND_TCGEN05, "split": sk.SKINNY_BACKEND_SPLITK}


def bound(depth, size, out=None):
    err = (1e-5 + max(0, depth - 32768) * 2.0 ** -32) * size
    return err if out is None else err + 2.0 ** -8 * (out.abs() + err)     # and a rounding to bf16


def terms(kind, rows, depth, seed):
    """Positive bf16: random, or the same everywhere (whose adds may all be rounded to one side)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "random":
        return torch.rand((rows, depth), generator=g, device="cuda").add_(0.01).bfloat16()
    return torch.full((rows, depth), float(kind), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("M,K", [(1, 32768), (20, 32768), (40, 32768), (300, 32768), (1, 300001), (17, 262144), (100, 300000),
                                 (1, 1 << 20), (20, 1 << 20), (64, 1 << 20), (130, 1 << 20)])
@pytest.mark.parametrize("kind", ["random", "1.0078125", "1.3359375", "1.9921875"])
def test_forward(kind, M, K, kernel):
    x, w = terms(kind, M, K, 1), terms(kind, 72, K, 2)
    y = torch.empty((M, 72), dtype=torch.float32, device="cuda")
    with sk.options(backend=KERNELS[kernel]):
        sk.linear(x, w, out=y)
    want = x.double() @ w.double().t()
    assert ((y.double() - want).abs() <= bound(K, want)).all(), ((y.double() - want).abs() / want).max().item()


@pytest.mark.parametrize("M", [2049, 32768, 100003, 1000003])
@pytest.mark.parametrize("kind", ["random", "1.0078125", "1.3359375"])
def test_bias_gradient(kind, M):
    dy = terms(kind, M, 24, 3)
    x, w = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda"), torch.zeros((24, 8), dtype=torch.bfloat16, device="cuda")
    db = sk.linear_grad(dy, x, w, input_grad=False, weight_grad=False, bias_grad=True)[2]
    want = dy.double().sum(0)
    assert ((db.double() - want).abs() <= bound(M, want)).all(), ((db.double() - want).abs() / want).max().item()


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("M,N,K", [(100003, 72, 136), (7, 300000, 64), (300, 100000, 72)])
@pytest.mark.parametrize("kind", ["random", "1.3359375"])
def test_products_of_the_backward_pass(kind, M, N, K, kernel):
    dy, x, w = terms(kind, M, N, 4), terms(kind, M, K, 5), terms(kind, N, K, 6)
    with sk.options(backend=KERNELS[kernel]):
        dx, dw, _ = sk.linear_grad(dy, x, w)
    for got, want, depth in ((dx, dy.double() @ w.double(), N), (dw, dy.double().t() @ x.double(), M)):
        assert ((got.double() - want).abs() <= bound(depth, want, want)).all()
