"""Gradients behind an activation by their norms: the elementwise bounds charge every dZ a full rounding, and over
many tokens would not notice a lost part of the depth.

The bound of a product's relative error in the Frobenius norm: dZ's rounding to bf16 is 2^-8 of each element at
most, and against factors of random sign its square adds up as the product's own does, so 2^-8; the product's own
rounding is 2^-8 of each element; the sums 1e-5 and dZ's fp32 steps below 2^-11 of a rounding: 2.1 2^-8 together."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk
import layer_ref as ref

pytestmark = pytest.mark.gpu

KERNELS = {"any": 0, "pair": sk.SKINNY_BACKEND_TCGEN05, "split": sk.SKINNY_BACKEND_SPLITK}
BOUND = 2.1 * 2.0 ** -8


def off(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


def case(M, N, K, act, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = 2 * N if act in ref.GATED else N
    return (torch.randn((M, N), generator=g, device="cuda").bfloat16(), torch.randn((M, K), generator=g, device="cuda").bfloat16(),
            torch.randn((rows, K), generator=g, device="cuda").bfloat16(),
            (2 * torch.randn((M, rows), generator=g, device="cuda")).bfloat16())


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("M,N,K", [(70001, 40, 72), (70001, 64, 64), (4103, 200, 264), (515, 512, 192), (1001, 67, 130),
                                   (129, 1024, 2048), (33, 61, 127), (1, 136, 72)])
def test_norms(M, N, K, act, kernel):
    dy, x, w, z = case(M, N, K, act, M + N)
    with sk.options(backend=KERNELS[kernel]):
        dx, dw, db = sk.linear_grad(dy, x, w, z, act, bias_grad=True)
    dz = ref.linear_dz(dy, z, act)
    xx, ww = x.double().cpu(), w.double().cpu()
    assert off(dx, dz @ ww) <= BOUND and off(dw, dz.t() @ xx) <= BOUND and off(db, dz.sum(0)) <= 1e-4
    if M > 64:      # it would notice a box of the depth that is left out, at either end
        assert off(dz[:-64].t() @ xx[:-64], dz.t() @ xx) > 2 * BOUND and off(dz[64:].t() @ xx[64:], dz.t() @ xx) > 2 * BOUND


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("M,N,K", [(70001, 40, 72), (4103, 200, 264), (1001, 67, 130), (300, 320, 512)])
def test_a_few_tokens_alone(M, N, K, act, kernel):
    """dY is zero but for some tokens, so the gradients are theirs alone."""
    dy, x, w, z = case(M, N, K, act, N)
    xx, ww = x.double().cpu(), w.double().cpu()
    for part in (slice(M - 1, M), slice(M - 17, M), slice(M - 65, M - 64), slice(0, 3), slice(M // 2, M // 2 + 64)):
        few = torch.zeros_like(dy)
        few[part] = dy[part]
        with sk.options(backend=KERNELS[kernel]):
            dx, dw, db = sk.linear_grad(few, x, w, z, act, bias_grad=True)
        dz = ref.linear_dz(dy[part], z[part], act)
        assert off(dx[part], dz @ ww) <= BOUND and off(dw, dz.t() @ xx[part]) <= BOUND and off(db, dz.sum(0)) <= 1e-4
        rest = dx.clone()
        rest[part] = 0
        assert not rest.any()


@pytest.mark.parametrize("M,N,K", [(70001, 40, 72), (515, 512, 192), (1001, 67, 130)])
def test_without_an_activation(M, N, K):
    """dZ is dY itself: one rounding alone."""
    dy, x, w, _ = case(M, N, K, None, K)
    dx, dw, _ = sk.linear_grad(dy, x, w)
    d, xx, ww = dy.double().cpu(), x.double().cpu(), w.double().cpu()
    assert off(dx, d @ ww) <= 1.05 * 2.0 ** -8 and off(dw, d.t() @ xx) <= 1.05 * 2.0 ** -8
