"""GPU parity of the experts' products against the plain 64-bit form: each sum
of products within 1e-5 of the sum of the magnitudes (the bound the library
keeps everywhere), then one rounding to the stored type."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import latency_skinny_bf16_gb300 as sk

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _init():
    assert sk.skinny_init(0) == sk.SKINNY_OK
    yield
    assert sk.skinny_get_device_status() == 0


@pytest.fixture(params=["auto", "tcgen05", "mma"])
def kernel(request):
    """Each kernel by force, where it takes the case, and the library's own choice."""
    force = {"auto": sk.SKINNY_BACKEND_AUTO, "tcgen05": sk.SKINNY_BACKEND_TCGEN05, "mma": sk.SKINNY_BACKEND_DOTPROD}
    with sk.options(backend=force[request.param]):
        yield request.param


def aligned(K, pad=0, offset=0):
    return K > 0 and (K + pad) % 8 == 0 and offset % 8 == 0


def stack(shape, ld, seed, scale=1.0, offset=0, same_sign=False):
    """A random bf16 CUDA stack [n, rows, cols] with row stride ld, its first element `offset` past an aligned one."""
    g = torch.Generator().manual_seed(seed)
    n, rows, cols = shape
    v = torch.randn(shape, generator=g) * scale
    buf = torch.full((n * rows * ld + offset + 8,), 3.0, dtype=torch.bfloat16)
    t = torch.as_strided(buf, shape, (rows * ld, ld, 1), offset)
    t.copy_((v.abs() if same_sign else v).bfloat16())
    return torch.as_strided(buf.cuda(), shape, (rows * ld, ld, 1), offset)


def host(t):
    return t.double().cpu().numpy()


def run(counts, N, K, act=None, out="fp32", pad=0, offset=0, extra=3, seed=0, same_sign=False, ypad=0):
    E, n = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = n + extra
    xs = stack((1, rows, K), K + pad, seed + 1, offset=offset, same_sign=same_sign)[0]
    w = stack((E, N * (2 if act else 1), K), K + pad, seed + 2, K ** -0.5, offset=offset, same_sign=same_sign)
    if extra:
        xs[n:] = float("nan")                  # rows no expert owns
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")                # experts without rows are not used
    y = torch.full((rows, N + ypad), -7.0, dtype=DT[out], device="cuda")
    sk.experts_gemm(xs, torch.from_numpy(off).cuda(), w, out=y[:, :N], activation=act)
    torch.cuda.synchronize()
    want, err = ref.experts(host(xs), off, host(w), bool(act))
    got = host(y)
    assert (got[n:] == -7.0).all() and (got[:, N:] == -7.0).all()
    bad = np.abs(got[:n, :N] - want[:n]) > ref.rounded(want[:n], err[:n], out)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[:n, :N][bad][0]} for {want[:n][bad][0]}"
    return xs, off, w, y


RAGGED = [0, 1, 16, 17, 0, 33, 64, 65, 2, 0]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 64), (8, 65), (100, 1000), (130, 1001), (64, 258), (300, 100), (129, 2880),
                                 (16, 7168), (1000, 72)])
def test_ragged(N, K, act, out, kernel):
    if kernel == "tcgen05" and not aligned(K):
        pytest.skip("rows not 16-byte aligned")
    run(RAGGED, N, K, act, out, seed=N + K)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (4, 4), (2, 0), (1, 0), (0, 1), (3, 5)])
def test_strides_and_alignment(pad, offset, act, kernel):
    if kernel == "tcgen05" and not aligned(136, pad, offset):
        with pytest.raises(sk.SkinnyError):
            run([3, 0, 20, 1], 72, 136, act, "bf16", pad=pad, offset=offset, ypad=5)
        return
    run([3, 0, 20, 1], 72, 136, act, "bf16", pad=pad, offset=offset, ypad=5)


@pytest.mark.parametrize("counts", [[0, 0, 0], [1], [0, 0, 1], [130, 0, 300], [8] * 300, [1] * 64 + [0] * 960,
                                    [0] * 1023 + [5], [64, 64], [200]])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_distributions(counts, act, kernel):
    run(counts, 40, 192, act, "fp32")


@pytest.mark.parametrize("N,K", [(4096, 512), (2112, 1536), (24, 8192), (5000, 128)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_larger(N, K, act, kernel):
    run([2, 0, 9, 1, 0, 40, 3], N, K, act, "bf16", seed=N)


@pytest.mark.parametrize("K", [2880, 7168, 14336])
def test_same_sign_operands(K, kernel):
    """Every product positive: rounding errors do not cancel."""
    run([1, 17, 0, 40], 136, K, None, "fp32", same_sign=True)


def test_not_finite_stays_in_its_row(kernel):
    xs, off, w, _ = run([5, 11, 3], 48, 128, None, "fp32")
    xs[2, 7], xs[9, 100], w[2, 5, 3] = float("nan"), float("inf"), float("nan")
    y = torch.zeros((xs.shape[0], 48), device="cuda")
    sk.experts_gemm(xs, torch.from_numpy(off).cuda(), w, out=y)
    y = y.cpu().numpy()
    assert np.isnan(y[2]).all() and not np.isfinite(y[9]).any()
    assert np.isnan(y[16:19, 5]).all()
    rest = np.delete(np.arange(19), [2, 9, 16, 17, 18])
    assert np.isfinite(y[rest]).all() and np.isfinite(np.delete(y[16:19], 5, axis=1)).all()


def test_swiglu_far_gates(kernel):
    """Gates far from zero: SiLU tends to 0 on the left, to its argument on the right."""
    w = torch.zeros((1, 4, 8), dtype=torch.bfloat16, device="cuda")
    w[0, 0, 0], w[0, 1, 0], w[0, 2, 1], w[0, 3, 1] = -1.0, 1.0, 1.0, 1.0
    xs = torch.zeros((3, 8), dtype=torch.bfloat16, device="cuda")
    xs[:, 0] = torch.tensor([50.0, 200.0, 1e30])
    xs[:, 1] = 2.0
    y = sk.experts_gemm(xs, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), w,
                        out=torch.empty((3, 2), device="cuda"), activation="swiglu").cpu().numpy()
    assert (np.abs(y[:, 0]) < 1e-15).all()
    x0 = xs[:, 0].double().cpu().numpy()
    assert (np.abs(y[:, 1] - 2 * x0) <= 1e-6 * x0).all()


def test_offsets_are_clamped_to_the_rows(kernel):
    """Offsets past the rows, negative or falling are cut: nothing outside the rows is read or written."""
    xs, w = stack((1, 6, 64), 64, 1)[0], stack((4, 32, 64), 64, 2)
    y = torch.full((8, 32), -7.0, device="cuda")
    off = torch.tensor([-3, 2, 100, 50, 1 << 30], dtype=torch.int32, device="cuda")
    sk.experts_gemm(xs, off, w, out=y[:6])
    torch.cuda.synchronize()
    assert (y[6:] == -7.0).all()
    want = np.concatenate([host(xs[:2]) @ host(w[0]).T, host(xs[2:]) @ host(w[1]).T])
    assert np.abs(host(y[:6]) - want).max() < 1e-2


def test_empty_calls_and_k_zero():
    w = torch.zeros((2, 8, 0), dtype=torch.bfloat16, device="cuda")
    y = torch.full((3, 8), -7.0, device="cuda")
    sk.experts_gemm(torch.zeros((3, 0), dtype=torch.bfloat16, device="cuda"),
                    torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), w, out=y)
    assert (y[:2] == 0).all() and (y[2:] == -7.0).all()
    out = sk.experts_gemm(torch.zeros((0, 8), dtype=torch.bfloat16, device="cuda"),
                          torch.zeros(3, dtype=torch.int32, device="cuda"),
                          torch.zeros((2, 8, 8), dtype=torch.bfloat16, device="cuda"))
    assert tuple(out.shape) == (0, 8)


@pytest.mark.parametrize("K", [256, 255])
def test_graph_streams_and_repeats(K, kernel):
    """Bits repeat from run to run, under PDL, in a graph whose inputs change, and on a given stream."""
    if kernel == "tcgen05" and not aligned(K):
        pytest.skip("rows not 16-byte aligned")
    counts = [[3, 0, 20, 1], [0, 9, 0, 15]]
    xs, w = stack((1, 24, K), K, 1)[0], stack((4, 96, K), K, 2, 0.1)
    off = [torch.tensor([0] + list(np.cumsum(c)), dtype=torch.int32, device="cuda") for c in counts]
    offsets = off[0].clone()
    want = [sk.experts_gemm(xs, o, w, activation="swiglu") for o in off]
    for pdl in (0, 1):
        with sk.options(pdl=pdl):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            got = sk.experts_gemm(xs, off[1], w, activation="swiglu", stream=s)
            s.synchronize()
            assert torch.equal(got, want[1])
            y = torch.empty_like(want[0])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                sk.experts_gemm(xs, offsets, w, out=y, activation="swiglu")
            for o, v in zip(off, want):
                offsets.copy_(o)
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(y, v)
            del g


def test_weights_past_32_bits(kernel):
    """Experts whose byte offsets pass 2^32."""
    E, N, K = 40, 8192, 8192                 # 5.4 GB
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[0, :, 1] = 1.0
    w[E - 1, :, 3] = torch.arange(N, device="cuda") % 128
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = 2
    off[E] = 5
    xs = torch.zeros((5, K), dtype=torch.bfloat16, device="cuda")
    xs[:, 1], xs[:, 3] = 2.0, torch.arange(5, device="cuda")
    y = sk.experts_gemm(xs, off, w, out=torch.empty((5, N), device="cuda"))
    assert (y[:2] == 2.0).all()
    assert torch.equal(y[2:], torch.arange(2, 5, device="cuda")[:, None] * (torch.arange(N, device="cuda") % 128).float())


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_bounded_waits_report_and_recover(act):
    """A wait without any budget gives up at once, the status says so, and the next call is right."""
    with sk.options(backend=sk.SKINNY_BACKEND_TCGEN05):
        xs, off, w, _ = run([3, 0, 20, 1], 200, 640, act, "fp32")
        offsets = torch.from_numpy(off).cuda()
        want = sk.experts_gemm(xs, offsets, w, activation=act)
        with sk.options(wait_timeout_us=0):
            sk.experts_gemm(xs, offsets, w, activation=act)
            torch.cuda.synchronize()
        assert sk.skinny_get_device_status() & 0xFF == sk.SKINNY_ERR_DEVICE_TIMEOUT
        n = int(off[-1])
        for _ in range(3):
            assert torch.equal(sk.experts_gemm(xs, offsets, w, activation=act)[:n], want[:n])
        assert sk.skinny_get_device_status() == 0


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("N,K", [(5, 63), (3, 7), (2, 9), (8, 1), (8, 3), (77, 130), (77, 129), (104, 777), (264, 57),
                                 (136, 1001), (40, 514), (40, 2052), (300, 6121)])
@pytest.mark.parametrize("counts", [[1, 0, 2], [0, 1, 16, 17, 33, 65]])
def test_rows_that_lie_alike(N, K, counts, act):
    """Odd lengths: rows of W that start alike within 16 bytes share a tile, also where N is no multiple of
    their distance, or less than it."""
    run(counts, N, K, act, "fp32", seed=N * K)


@pytest.mark.parametrize("K,ld", [(129, 129), (130, 130), (132, 140), (250, 251)])
def test_infinities_of_neighbouring_rows_and_padding(K, ld):
    """What lies before and behind a row of W or X, within the 16 bytes of its ends, does not reach its sums."""
    E, N, rows = 2, 48, 7
    w, xs = stack((E, N, K), ld, 1), stack((1, rows, K), ld, 2)[0]
    off = torch.tensor([0, 4, rows], dtype=torch.int32, device="cuda")
    want = sk.experts_gemm(xs, off, w, out=torch.empty((rows, N), device="cuda")).clone()
    bad = [(0, 5), (0, 11), (1, 0), (1, N - 1)]
    for e, n in bad:
        w[e, n, 0], w[e, n, K - 1] = float("inf"), float("nan")
    xs[2, 0], xs[2, K - 1] = float("nan"), float("inf")
    if ld > K:
        torch.as_strided(w, (E * N - 1, ld - K), (ld, 1), w.storage_offset() + K).fill_(float("nan"))
        torch.as_strided(xs, (rows - 1, ld - K), (ld, 1), xs.storage_offset() + K).fill_(float("inf"))
    got = sk.experts_gemm(xs, off, w, out=torch.empty((rows, N), device="cuda"))
    hit = torch.zeros((rows, N), dtype=torch.bool, device="cuda")
    for e, n in bad:
        hit[:4, n] |= e == 0
        hit[4:, n] |= e == 1
    hit[2] = True
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("N,K,act", [(6000, 1001, None), (6008, 1001, "swiglu"), (6007, 1001, None), (9001, 130, None), (9002, 258, "swiglu")])
def test_long_lines_of_unaligned_rows(N, K, act):
    """Tens of rows an expert and long lines of odd rows, whose last tiles are in part empty."""
    run([33, 0, 9, 64, 40], N, K, act, "bf16", seed=N)
