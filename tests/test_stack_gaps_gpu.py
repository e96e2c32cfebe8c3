"""Stacks whose matrices lie further apart than their rows need: the stride of
an expert or an adapter is any number of elements, what lies between the
matrices and between their rows is NaN, and none of it reaches a result."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import latency_skinny_bf16_gb300 as sk
import test_lora_gpu
from test_experts_gemm_gpu import host, kernel  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _init():
    assert sk.skinny_init(0) == sk.SKINNY_OK
    yield
    assert sk.skinny_get_device_status() == 0


def stack(n, rows, cols, ld, gap, seed, scale=1.0, offset=0):
    """Random bf16 [n, rows, cols], row stride ld, matrix stride rows * ld + gap, NaN wherever no element lies."""
    g = torch.Generator().manual_seed(seed)
    lde = rows * ld + gap
    buf = torch.full((n * lde + offset + 8,), float("nan"), dtype=torch.bfloat16)
    torch.as_strided(buf, (n, rows, cols), (lde, ld, 1), offset).copy_((torch.randn(n, rows, cols, generator=g) * scale).bfloat16())
    return torch.as_strided(buf.cuda(), (n, rows, cols), (lde, ld, 1), offset)


GAPS = [8, 4, 1, 4104, 1001]


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("N,K,pad,offset", [(48, 136, 0, 0), (72, 128, 8, 8), (33, 320, 0, 0), (40, 129, 0, 0), (20, 258, 2, 1)])
@pytest.mark.parametrize("gap", GAPS)
def test_experts(N, K, pad, offset, gap, act, kernel):  # noqa: F811
    counts = [0, 3, 1, 0, 40, 17, 2]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows, E = int(off[-1]) + 2, len(counts)
    xs = stack(1, rows, K, K + pad, 0, 1, offset=offset)[0]
    w = stack(E, N * (2 if act else 1), K, K + pad, gap, 2, K ** -0.5, offset)
    xs[rows - 2:], w[0], w[3] = float("nan"), float("nan"), float("nan")
    y = torch.full((rows, N + 1), -7.0, device="cuda")

    def call():
        sk.experts_gemm(xs, torch.from_numpy(off).cuda(), w, out=y[:, :N], activation=act)
        torch.cuda.synchronize()

    if kernel == "tcgen05" and any(v % 8 for v in (K + pad, offset, gap)):
        with pytest.raises(sk.SkinnyError):
            call()
        return
    call()
    want, err = ref.experts(host(xs), off, host(w), bool(act))
    got, n = host(y), int(off[-1])
    assert (got[n:] == -7.0).all() and (got[:, N:] == -7.0).all()
    assert (np.abs(got[:n, :N] - want[:n]) <= ref.rounded(want[:n], err[:n], "fp32")).all()


@pytest.mark.parametrize("K", [1536, 1535])
@pytest.mark.parametrize("gap", [8, 3])
def test_experts_long_lines(K, gap, kernel):  # noqa: F811
    """Enough rows and lines for the kernels that the library chooses on large calls."""
    counts = [20, 0, 33, 9]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xs, w = stack(1, 62, K, K, 0, 1)[0], stack(4, 6000, K, K, gap, 2, K ** -0.5)
    if kernel == "tcgen05" and (K % 8 or gap % 8):
        pytest.skip("rows not 16-byte aligned")
    y = sk.experts_gemm(xs, torch.from_numpy(off).cuda(), w, out=torch.empty((62, 6000), device="cuda"))
    want, err = ref.experts(host(xs), off, host(w), False)
    assert (np.abs(host(y) - want) <= ref.rounded(want, err, "fp32")).all()


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("N,K,R,pad,offset", [(200, 264, 16, 0, 0), (136, 256, 64, 8, 8), (65, 129, 24, 0, 0), (100, 130, 33, 3, 1)])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("M", [5, 40])
def test_adapters(N, K, R, pad, offset, gap, M, out):
    L = 5
    x, w = stack(1, M, K, K + pad, 0, 1, offset=offset)[0], stack(1, N, K, K + pad, 0, 2, K ** -0.5, offset)[0]
    a, b = stack(L, R, K, K + pad, gap, 3, K ** -0.5, offset), stack(L, N, R, R + pad, gap, 4, R ** -0.5, offset)
    ranks = np.array([R, max(1, R // 2), 0, 1, R], np.int32)
    scales = np.linspace(0.5, 2.0, L).astype(np.float32)
    ids = np.random.default_rng(M).integers(-1, L, M).astype(np.int32)
    ids[:3] = [L - 1, 0, 1]                    # the last adapter's last row is used
    test_lora_gpu.check(x, w, a, b, ids, ranks, scales, out, ypad=1)


def test_one_matrix_needs_no_stride():
    w = stack(1, 48, 64, 64, 0, 1)
    xs = stack(1, 9, 64, 64, 0, 2)[0]
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    view = torch.as_strided(w, (1, 48, 64), (1, 64, 1), 0)
    assert torch.equal(sk.experts_gemm(xs, off, view), sk.experts_gemm(xs, off, w))
