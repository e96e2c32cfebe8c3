"""GPU parity of the projection with low-rank adapters against the plain
64-bit form; the error bound is derived in experts_ref.lora."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import latency_skinny_bf16_gb300 as sk
from test_experts_gemm_gpu import DT, host, stack

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _init():
    assert sk.skinny_init(0) == sk.SKINNY_OK
    yield
    assert sk.skinny_get_device_status() == 0


def inputs(M, N, K, L, R, seed=0, pad=0, offset=0, mixed=True):
    rng = np.random.default_rng(seed)
    x, w = stack((1, M, K), K + pad, seed + 1, offset=offset)[0], stack((1, N, K), K + pad, seed + 2, K ** -0.5, offset)[0]
    a, b = stack((L, R, K), K + pad, seed + 3, K ** -0.5, offset), stack((L, N, R), R + pad, seed + 4, R ** -0.5, offset)
    ranks = rng.integers(0, R + 1, L).astype(np.int32) if mixed else np.full(L, R, np.int32)
    ranks[0] = R
    scales = (0.5 + rng.random(L)).astype(np.float32)
    return x, w, a, b, ranks, scales


def check(x, w, a, b, ids, ranks, scales, out="fp32", ypad=0):
    M, N = x.shape[0], w.shape[0]
    if ranks is not None:
        for i, r in enumerate(ranks):          # what lies past an adapter's rank is not used
            a[i, max(0, int(r)):] = float("nan")
            b[i, :, max(0, int(r)):] = float("nan")
    y = torch.full((M, N + ypad), -7.0, dtype=DT[out], device="cuda")
    dev = [None if v is None else torch.from_numpy(v).cuda() for v in (ids, ranks, scales)]
    sk.lora_gemm(x, w, a, b, *dev, out=y[:, :N])
    torch.cuda.synchronize()
    want, err = ref.lora(host(x), host(w), host(a), host(b), ids, ranks, scales)
    got = host(y)
    assert (got[:, N:] == -7.0).all()
    bad = np.abs(got[:, :N] - want) > ref.rounded(want, err, out) + 1e-6
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}"
    return y


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K,L,R", [
    (1, 2112, 7168, 8, 16), (1, 1, 8, 1, 1), (2, 33, 100, 3, 4), (5, 128, 64, 2, 8), (16, 1000, 1536, 6, 64),
    (9, 257, 1001, 4, 24), (3, 100, 258, 3, 3), (8, 129, 520, 4, 128), (12, 130, 776, 5, 256), (7, 64, 72, 30, 33)])
def test_shapes(M, N, K, L, R, out):
    x, w, a, b, ranks, scales = inputs(M, N, K, L, R, seed=M + N)
    ids = np.random.default_rng(K).integers(-1, L, M).astype(np.int32)
    check(x, w, a, b, ids, ranks, scales, out, ypad=3)


@pytest.mark.parametrize("M,L", [(17, 3), (33, 40), (64, 1), (64, 64), (64, 9)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_many_tokens(M, L, out):
    x, w, a, b, ranks, scales = inputs(M, 512, 256, L, 32, seed=M + L)
    ids = np.random.default_rng(L).integers(-1, L, M).astype(np.int32)
    check(x, w, a, b, ids, ranks, scales, out)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "out of range", "one adapter", "own adapters", "zero ranks", "ranks out of range"])
def test_special_ids(kind, out):
    M, L, R = 13, 16, 16
    x, w, a, b, ranks, scales = inputs(M, 200, 320, L, R, seed=3)
    ids = np.arange(M, dtype=np.int32)
    if kind == "none":
        ids[:] = -1
    elif kind == "out of range":
        ids[::2] = L
        ids[1] = np.iinfo(np.int32).min
        ids[3] = np.iinfo(np.int32).max
    elif kind == "one adapter":
        ids[:] = 5
    elif kind == "zero ranks":
        ranks[:] = 0
    elif kind == "ranks out of range":
        ranks[:8], ranks[8:] = R + 100, -4
    check(x, w, a, b, ids, ranks, scales, out)


@pytest.mark.parametrize("pad,offset", [(8, 0), (4, 4), (2, 2), (1, 0), (0, 1), (8, 8)])
def test_strides_and_alignment(pad, offset):
    x, w, a, b, ranks, scales = inputs(6, 136, 264, 4, 16, seed=9, pad=pad, offset=offset)
    check(x, w, a, b, np.array([0, 3, -1, 3, 1, 2], np.int32), ranks, scales, "bf16", ypad=1)


def test_without_ranks_and_scales():
    x, w, a, b, _, _ = inputs(6, 136, 264, 4, 16, seed=9)
    check(x, w, a, b, np.array([0, 3, -1, 3, 1, 2], np.int32), None, None)


@pytest.mark.parametrize("L,R", [(0, 8), (4, 0)])
def test_no_adapters_is_the_projection(L, R):
    x, w = stack((1, 5, 256), 256, 1)[0], stack((1, 96, 256), 256, 2)[0]
    a, b = torch.zeros((L, R, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((L, 96, R), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert torch.equal(sk.lora_gemm(x, w, a, b, ids), sk.gemm(x, w))


def test_tokens_without_adapter_keep_the_projection():
    x, w, a, b, ranks, scales = inputs(10, 300, 512, 4, 16, seed=5)
    ids = np.array([-1, 0, -1, 1, 2, -1, 3, 9, -5, 0], np.int32)
    y = check(x, w, a, b, ids, ranks, scales)
    none = (ids < 0) | (ids >= 4)
    base = sk.gemm(x, w)
    assert torch.equal(y[none], base[none])


def test_not_finite_stays_with_its_adapter():
    x, w, a, b, ranks, scales = inputs(4, 64, 128, 3, 8, seed=6, mixed=False)
    a[1, 2, 5] = float("nan")
    b[2, 7, 1] = float("inf")
    y = sk.lora_gemm(x, w, a, b, torch.tensor([0, 1, 2, -1], dtype=torch.int32, device="cuda")).cpu().numpy()
    assert np.isfinite(y[[0, 3]]).all() and np.isnan(y[1]).all()
    assert not np.isfinite(y[2, 7]) and np.isfinite(np.delete(y[2], 7)).all()


@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_graph_and_streams(out):
    x, w, a, b, ranks, scales = inputs(16, 640, 1024, 6, 32, seed=8)
    cases = [np.random.default_rng(s).integers(-1, 6, 16).astype(np.int32) for s in (1, 2)]
    rk, sc = torch.from_numpy(ranks).cuda(), torch.from_numpy(scales).cuda()
    ids = torch.zeros(16, dtype=torch.int32, device="cuda")
    for pdl in (0, 1, 2):
        with sk.options(pdl=pdl):
            want = []
            for c in cases:
                ids.copy_(torch.from_numpy(c))
                want.append(check(x.clone(), w, a, b, c, ranks, scales, out))
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            y = torch.empty((16, 640), dtype=DT[out], device="cuda")
            ws = torch.empty(sk.lora_workspace(16, 640, 32, DT[out]), dtype=torch.uint8, device="cuda")
            sk.lora_gemm(x, w, a, b, ids, rk, sc, out=y, workspace=ws, stream=s)
            s.synchronize()
            assert torch.equal(y, want[1])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                for _ in range(3):
                    sk.lora_gemm(x, w, a, b, ids, rk, sc, out=y, workspace=ws)
            for c, v in zip(cases, want):
                ids.copy_(torch.from_numpy(c))
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(y, v)
            del g


def test_infinite_adapter_gives_what_the_definition_gives():
    """An infinite element of B: its product with V is infinite of V's sign (NaN where V is 0), whatever bits V has."""
    x, w, a, b, _, _ = inputs(9, 64, 128, 3, 8, seed=6, mixed=False)
    x[3] = 0.0                                              # V of this token is 0
    b[:, 7, 1], b[:, 9, 2] = float("inf"), float("-inf")
    ids = torch.arange(9, dtype=torch.int32, device="cuda") % 3
    y = sk.lora_gemm(x, w, a, b, ids).double().cpu().numpy()
    want = np.stack([host(w) @ host(x)[m] + host(b)[m % 3] @ (host(a)[m % 3] @ host(x)[m]) for m in range(9)])
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.isnan(want[3, 7])
    inf = np.isinf(want)
    assert inf.sum() == 16 and np.array_equal(y[inf], want[inf]) and np.isfinite(y[~inf & ~np.isnan(want)]).all()
