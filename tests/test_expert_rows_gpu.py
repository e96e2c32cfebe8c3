"""GPU parity of dispatch, combine and combine's gradient against plain 64-bit
forms.  Whole numbers and copied rows must be equal.  A sum of n products in
fp32 with one rounding per multiply-add is within n * 2^-24 * (sum of the
magnitudes) to first order (1% is allowed for the higher ones); the stored
type adds half a step of its own."""
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


def matrix(rows, cols, dtype, seed, pad=0, offset=0):
    """A random CUDA matrix, its row stride `pad` above its width, its first element `offset` past an aligned one."""
    g = torch.Generator().manual_seed(seed)
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 8,), 7.0, dtype=DT[dtype])
    t = torch.as_strided(buf, (rows, cols), (ld, 1), offset)
    t.copy_(torch.randn(rows, cols, generator=g).to(DT[dtype]))
    buf = buf.cuda()
    return torch.as_strided(buf, (rows, cols), (ld, 1), offset)


def host(t):
    return t.double().cpu().numpy()


def check_dispatch(ids, E, x, out):
    xs, pos, order, offsets = out
    rpos, rorder, roff = ref.dispatch(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), roff)
    assert np.array_equal(pos.cpu().numpy(), rpos)
    assert np.array_equal(order.cpu().numpy(), rorder)
    n = int(roff[-1])
    if x is not None:
        k = ids.shape[1]
        got, want = xs[:n].float().cpu(), x.float().cpu()[torch.from_numpy(rorder[:n].astype(np.int64)) // max(k, 1)]
        assert torch.equal(got, want)
    return n


@pytest.mark.parametrize("pdl", [0, 1])
@pytest.mark.parametrize("T,k,E,H,dtype,drop", [
    (1, 1, 1, 8, "bf16", 0), (1, 8, 256, 7168, "bf16", 0), (3, 2, 7, 33, "bf16", 0.3), (64, 8, 384, 2880, "bf16", 0.1),
    (61, 6, 64, 1001, "fp32", 0.5), (128, 8, 256, 64, "fp32", 0), (127, 64, 64, 24, "bf16", 0),
    (129, 8, 256, 96, "bf16", 0.1), (1000, 8, 256, 128, "bf16", 0.05), (5000, 4, 33, 12, "bf16", 0.5),
    (3000, 1, 8192, 4, "fp32", 0), (40, 64, 8192, 2, "bf16", 0.2), (70000, 2, 16, 3, "fp32", 0.01)])
def test_dispatch(T, k, E, H, dtype, drop, pdl):
    ids, _ = ref.routing(T, k, min(E, 512), seed=T + E, drop=drop, skew=1.0)
    x = matrix(T, H, dtype, seed=T)
    with sk.options(pdl=pdl):
        out = sk.expert_dispatch(torch.from_numpy(ids).cuda(), E, x=x)
        torch.cuda.synchronize()
    check_dispatch(ids, E, x, out)


@pytest.mark.parametrize("T,k", [(5, 3), (700, 5)])
@pytest.mark.parametrize("kind", ["all dropped", "one expert", "out of range", "repeated", "last expert"])
def test_dispatch_special_ids(T, k, kind):
    E = 40
    ids, _ = ref.routing(T, k, E, seed=5)
    if kind == "all dropped":
        ids[:] = -1
    elif kind == "one expert":
        ids[:] = 17
    elif kind == "out of range":
        ids[::2, 0] = E
        ids[1::2, 1] = np.iinfo(np.int32).min
        ids[::3, 2] = np.iinfo(np.int32).max
    elif kind == "repeated":
        ids[:, 1] = ids[:, 0]
    else:
        ids[:] = E - 1
    x = matrix(T, 16, "bf16", 1)
    check_dispatch(ids, E, x, sk.expert_dispatch(torch.from_numpy(ids).cuda(), E, x=x))


@pytest.mark.parametrize("T", [6, 900])
@pytest.mark.parametrize("H,dtype,pad,offset", [(64, "bf16", 3, 0), (64, "bf16", 8, 1), (63, "bf16", 1, 0),
                                                (10, "fp32", 2, 2), (64, "bf16", 4, 4), (31, "fp32", 0, 1)])
def test_dispatch_strides_and_gaps(T, H, dtype, pad, offset):
    k, E = 3, 12
    ids, _ = ref.routing(T, k, E, seed=9, drop=0.2)
    wide = torch.full((T, k + 2), 3, dtype=torch.int32, device="cuda")
    wide[:, :k] = torch.from_numpy(ids).cuda()
    x = matrix(T, H, dtype, 2, pad, offset)
    base = torch.full((T * k * (H + pad) + offset + 8,), -5.0, dtype=DT[dtype], device="cuda")
    xs = torch.as_strided(base, (T * k, H), (H + pad, 1), offset)
    n = check_dispatch(ids, E, x, sk.expert_dispatch(wide[:, :k], E, x=x, xs=xs))
    mask = torch.ones_like(base, dtype=torch.bool)
    torch.as_strided(mask, (T * k, H), (H + pad, 1), offset)[:n] = False
    assert (base[mask] == -5.0).all()       # gaps and rows without an entry stay as they were


@pytest.mark.parametrize("T,k,H", [(0, 4, 8), (4, 0, 8), (4, 2, 0), (0, 0, 0)])
def test_dispatch_empty(T, k, H):
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    offsets = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    _, pos, order, offsets = sk.expert_dispatch(ids, 5, x=x, offsets=offsets)
    torch.cuda.synchronize()
    check_dispatch(ids.cpu().numpy(), 5, None, (None, pos, order, offsets))


def test_dispatch_sort_only():
    ids, _ = ref.routing(50, 4, 20, seed=3, drop=0.1)
    out = sk.expert_dispatch(torch.from_numpy(ids).cuda(), 20)
    assert out[0] is None
    check_dispatch(ids, 20, None, out)


COMBINE = [
    (1, 8, 256, 7168, "fp32", "bf16", 0.0), (64, 8, 256, 2880, "bf16", "bf16", 0.0), (7, 3, 9, 33, "bf16", "fp32", 0.3),
    (300, 6, 64, 1001, "fp32", "fp32", 0.5), (33, 9, 16, 40, "fp32", "bf16", 0.1), (5, 17, 32, 64, "bf16", "bf16", 0.0),
    (4, 64, 64, 12, "fp32", "bf16", 0.0), (2, 1, 4, 1, "bf16", "bf16", 0.0), (700, 2, 8, 24, "bf16", "bf16", 0.9)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,H,it,ot,drop", COMBINE)
def test_combine(T, k, E, H, it, ot, drop, weighted):
    ids, w = ref.routing(T, k, E, seed=H, drop=drop)
    pos, _, off = ref.dispatch(ids, E)
    w = w - 0.3
    w[pos < 0] = np.nan                       # the weight of a dropped entry is not used
    ys = matrix(T * k, H, it, seed=H + 1)
    if int(off[-1]) < T * k:
        ys[int(off[-1]):] = float("nan")      # nor are rows that no entry names
    out = torch.full((T, H + 3), -9.0, dtype=DT[ot], device="cuda")
    pt, wt = torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda() if weighted else None
    got = sk.expert_combine(ys, pt, wt, out=out[:, :H])
    torch.cuda.synchronize()
    y, mag = ref.combine(host(ys), pos, w if weighted else None)
    err = 1.01 * k * ref.U32 * mag
    assert (np.abs(host(got) - y) <= ref.rounded(y, err, ot)).all()
    assert (out[:, H:] == -9.0).all()
    again = sk.expert_combine(ys, pt, wt, out=torch.empty((T, H), dtype=DT[ot], device="cuda"))
    assert torch.equal(again, got)            # another alignment, the same sums in the same order


def test_combine_no_entries_and_bad_positions():
    ys = matrix(4, 16, "bf16", 1)
    pos = torch.tensor([[-1, -1], [4, 1 << 30], [-(1 << 31), 2]], dtype=torch.int32, device="cuda")
    got = sk.expert_combine(ys, pos, torch.ones((3, 2), device="cuda"))
    assert (got[:2] == 0).all() and torch.equal(got[2], ys[2])
    none = sk.expert_combine(ys, torch.zeros((3, 0), dtype=torch.int32, device="cuda"), out=torch.ones((3, 16), device="cuda"))
    assert (none == 0).all()


def test_combine_not_finite():
    """Infinities and NaN of live entries come through; a row of its own keeps them to itself."""
    ys = torch.ones((4, 8), device="cuda")
    ys[0, 1], ys[1, 2], ys[2, 3] = float("inf"), float("-inf"), float("nan")
    pos = torch.tensor([[0, 1], [2, 3], [3, -1]], dtype=torch.int32, device="cuda")
    got = sk.expert_combine(ys, pos, torch.full((3, 2), 0.5, device="cuda")).cpu().numpy()
    assert got[0, 1] == np.inf and got[0, 2] == -np.inf and np.isnan(got[1, 3])
    assert np.isfinite(got).sum() == got.size - 3 and (got[2] == 0.5).all()


GRAD = [(1, 8, 256, 7168, "bf16", 0.0), (64, 8, 64, 1001, "fp32", 0.1), (9, 3, 5, 33, "bf16", 0.4), (3, 17, 32, 64, "fp32", 0.0),
        (200, 6, 12, 520, "bf16", 0.0), (5, 64, 64, 8, "bf16", 0.1), (2, 1, 3, 1, "fp32", 0.0)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,H,dt,drop", GRAD)
def test_combine_grad(T, k, E, H, dt, drop, weighted):
    ids, w = ref.routing(T, k, E, seed=H, drop=drop)
    pos, _, off = ref.dispatch(ids, E)
    n = int(off[-1])
    w = w - 0.3
    w[pos < 0] = np.nan
    ys, dy = matrix(T * k, H, dt, seed=H + 1, pad=8), matrix(T, H, dt, seed=H + 2)
    ys[n:] = float("nan")
    dys = torch.full((T * k, H), -5.0, dtype=DT[dt], device="cuda")
    dw = torch.full((T, k + 1), -9.0, device="cuda")
    sk.expert_combine_grad(dy, ys, torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda() if weighted else None,
                           dys=dys, dweights=dw[:, :k])
    torch.cuda.synchronize()
    rys, rw, mag = ref.combine_grad(host(dy), host(ys), pos, w if weighted else None)
    got = host(dys)
    assert (got[n:] == -5.0).all()
    assert (np.abs(got[:n] - rys[:n]) <= ref.rounded(rys[:n], ref.U32 * np.abs(rys[:n]), dt)).all()
    chain = 8 * (H // 2048 + 1) + 5 + 8 if dt == "bf16" else 4 * (H // 1024 + 1) + 5 + 8
    chain = max(chain, H // 256 + 1 + 13)     # element by element: one in 256
    assert (np.abs(host(dw[:, :k]) - rw) <= 1.01 * chain * ref.U32 * mag + ref.TINY["fp32"]).all()
    assert (dw[:, k:] == -9.0).all()


def test_combine_grad_without_weight_gradient():
    ids, w = ref.routing(12, 4, 8, seed=1)
    pos, _, _ = ref.dispatch(ids, 8)
    dy = matrix(12, 64, "bf16", 3)
    pt, wt = torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda()
    full, _ = sk.expert_combine_grad(dy, matrix(48, 64, "bf16", 4), pt, wt)
    dys = torch.empty((48, 64), dtype=torch.bfloat16, device="cuda")
    assert sk.skinny_expert_combine_grad(dy.data_ptr(), 64, 0, 0, 48, pt.data_ptr(), wt.data_ptr(), 4, 12, 4, 64,
                                         sk.SKINNY_BF16, dys.data_ptr(), 64, 0, 0,
                                         torch.cuda.current_stream().cuda_stream) == sk.SKINNY_OK
    assert torch.equal(dys, full)


def test_gradients_against_differences():
    """combine is linear in its rows and in its weights, and dispatch in its
    rows: the change of <dy, y> along a direction is the gradient's product
    with it.  fp32 throughout; every product of the two sides is rounded a few
    times, so 64 * 2^-24 of the sum of the magnitudes covers both."""
    T, k, E, H = 20, 4, 9, 257
    ids, w = ref.routing(T, k, E, seed=2, drop=0.2)
    it = torch.from_numpy(ids).cuda()
    x = matrix(T, H, "fp32", 1)
    xs, pos, _, off = sk.expert_dispatch(it, E, x=x, xs=torch.zeros((T * k, H), device="cuda"))
    n = int(off[-1])
    wt, dy = torch.from_numpy(w).cuda(), matrix(T, H, "fp32", 3)
    dys, dw = sk.expert_combine_grad(dy, xs, pos, wt, dys=torch.zeros_like(xs))
    dx = sk.expert_combine(dys, pos)
    vy, vw, vx = matrix(T * k, H, "fp32", 5), matrix(T, k, "fp32", 6), matrix(T, H, "fp32", 7)

    def change(f, *at):
        a, b = f(+1), f(-1)
        d = dy.double()
        return float((d * (a.double() - b.double())).sum() / 2), float((d.abs() * (a.double().abs() + b.double().abs())).sum())

    for f, grad, v in ((lambda s: sk.expert_combine(xs + s * vy, pos, wt), dys, vy),
                       (lambda s: sk.expert_combine(xs, pos, wt + s * vw), dw, vw),
                       (lambda s: sk.expert_combine(sk.expert_dispatch(it, E, x=x + s * vx)[0], pos, wt), dx, vx)):
        got, mag = change(f)
        want = float((grad.double() * v.double()).sum())
        assert abs(got - want) <= 64 * ref.U32 * (mag + float((grad.double() * v.double()).abs().sum()))
    assert n > 0


@pytest.mark.parametrize("T", [40, 600])
def test_rows_in_a_graph_and_on_another_stream(T):
    """Dispatch, combine and the gradient captured together, with and without
    PDL, give the bits of the eager calls; new inputs in the same buffers are
    used by the replay."""
    k, E, H = 4, 24, 136
    x, dy = matrix(T, H, "bf16", 1), matrix(T, H, "bf16", 2)
    wt = torch.rand((T, k), device="cuda")
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    a = [torch.from_numpy(ref.routing(T, k, E, seed=s, drop=0.1)[0]).cuda() for s in (1, 2)]

    def step(stream=None):
        xs, pos, order, off = sk.expert_dispatch(ids, E, x=x, xs=torch.zeros((T * k, H), dtype=x.dtype, device="cuda"), stream=stream)
        y = sk.expert_combine(xs, pos, wt, stream=stream)
        dys, dw = sk.expert_combine_grad(dy, xs, pos, wt, dys=torch.zeros_like(xs), stream=stream)
        return [xs, pos, order, off, y, dys, dw, sk.expert_combine(dys, pos, stream=stream)]

    eager = []
    for i in a:
        ids.copy_(i)
        eager.append([t.clone() for t in step()])
    for pdl in (0, 1):
        with sk.options(pdl=pdl):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                ids.copy_(a[0])
                step()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = step()
            for i, want in zip(a, eager):
                ids.copy_(i)
                g.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(o, w) for o, w in zip(out, want))
            del g, out
    # a stream that is given, torch's own current one elsewhere
    ids.copy_(a[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, pos = None, None
    xs, pos, order, off = sk.expert_dispatch(ids, E, x=x, stream=s)
    y = sk.expert_combine(xs, pos, wt, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, eager[1][4])


def test_places_past_32_bits():
    """Rows whose byte offsets pass 2^32: the copies and sums land where they should."""
    T, k, E, H = 40000, 2, 4, 32768          # 5.2 GB of rows
    ids, _ = ref.routing(T, k, E, seed=8)
    x = torch.randn((T, H), device="cuda", dtype=torch.bfloat16)
    xs, pos, order, off = sk.expert_dispatch(torch.from_numpy(ids).cuda(), E, x=x)
    for f in (0, 1, T * k // 2, T * k - 1):
        p = int(pos.reshape(-1)[f])
        assert torch.equal(xs[p], x[f // k])
    assert torch.equal(xs[-1], x[int(order[-1]) // k])
    y = sk.expert_combine(xs, pos, torch.full((T, k), 0.5, device="cuda"))
    assert torch.equal(y, x)


@pytest.mark.parametrize("H,dtype", [(1030, "bf16"), (2051, "bf16"), (4097, "fp32"), (1, "fp32"), (3, "bf16")])
@pytest.mark.parametrize("k", [1, 8, 20])
def test_combine_rows_of_any_alignment(H, dtype, k):
    """Rows that start and end off 16 bytes, chunks of them, the first and the last row of a tensor that itself
    starts off 16 bytes, and rows that lie end to end with a stride above their width."""
    T, E = 11, 40
    ids, w = ref.routing(T, k, E, seed=H + k, drop=0.2)
    pos, _, _ = ref.dispatch(ids, E)
    pos[0, 0], pos[1, 0] = 0, T * k - 1
    pt, wt = torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda()
    for pad, offset in ((0, 0), (0, 1), (5, 3)):
        ys = matrix(T * k, H, dtype, seed=H, pad=pad, offset=offset)
        got = sk.expert_combine(ys, pt, wt)
        y, mag = ref.combine(host(ys), pos, w)
        assert (np.abs(host(got) - y) <= ref.rounded(y, 1.01 * k * ref.U32 * mag, dtype)).all()
        even = torch.zeros((T * k, H + 8 - H % 8), dtype=ys.dtype, device="cuda")[:, :H]
        even.copy_(ys)
        assert torch.equal(sk.expert_combine(even, pt, wt, out=torch.empty((T, H + 8 - H % 8), dtype=ys.dtype, device="cuda")[:, :H]), got)


def test_combine_bounded_wait_reports_and_recovers():
    ys = matrix(64, 1001, "fp32", seed=3)
    pos = torch.arange(64, dtype=torch.int32, device="cuda").reshape(16, 4)
    want = sk.expert_combine(ys, pos)
    with sk.options(wait_timeout_us=0):
        sk.expert_combine(ys, pos)
        torch.cuda.synchronize()
    assert sk.skinny_get_device_status() & 0xFF == sk.SKINNY_ERR_DEVICE_TIMEOUT
    for _ in range(3):
        assert torch.equal(sk.expert_combine(ys, pos), want)
    assert sk.skinny_get_device_status() == 0


@pytest.mark.parametrize("T,k,H,dtype", [(40, 8, 2881, "bf16"), (33, 1, 1, "bf16"), (64, 3, 7, "bf16"), (40, 20, 1017, "bf16"),
                                         (50, 2, 1016, "bf16"), (700, 2, 2051, "fp32"), (700, 6, 509, "fp32"), (640, 1, 1, "fp32"),
                                         (640, 9, 34, "fp32")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (5, 3)])
def test_combine_grad_rows_of_any_alignment(T, k, H, dtype, pad, offset):
    """Rows off 8 bytes: whole pieces and their ends; rows no entry names and the gaps between rows stay."""
    ids, w = ref.routing(T, k, max(40, k), seed=H + k, drop=0.2)
    pos, _, _ = ref.dispatch(ids, max(40, k))
    n = int((pos >= 0).sum())
    pos[pos == n - 1] = T * k - 1             # the last row of all, and one that no entry names
    ys, dy = matrix(T * k, H, dtype, H + 1, pad=pad, offset=offset), matrix(T, H, dtype, H + 2, pad=pad, offset=offset)
    pt, wt = torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda()
    ld = H + pad
    buf = torch.full((T * k * ld + offset + 16,), -5.0, dtype=DT[dtype], device="cuda")
    dys = torch.as_strided(buf, (T * k, H), (ld, 1), offset + 1)
    _, dw = sk.expert_combine_grad(dy, ys, pt, wt, dys=dys)
    rys, rw, mag = ref.combine_grad(host(dy), host(ys), pos, w)
    named = ~np.isnan(rys[:, 0])
    got = host(dys)
    assert (got[~named] == -5.0).all()
    assert (np.abs(got[named] - rys[named]) <= ref.rounded(rys[named], ref.U32 * np.abs(rys[named]), dtype)).all()
    # a lane adds four pieces of every 2032 bytes, a warp its lanes, four warps theirs
    el = 2 if dtype == "bf16" else 4
    chain = 4 * (16 // el) * ((H * el + 2031) // 2032) + 5 + 4
    chain = max(chain, H // 256 + 1 + 13)
    assert (np.abs(host(dw) - rw) <= 1.01 * chain * ref.U32 * mag + ref.TINY["fp32"]).all()
    dys.fill_(-5.0)
    assert (buf == -5.0).all()
    # without the weights' gradient the rows are the same
    sk.expert_combine_grad(dy, ys, pt, wt, dys=dys)
    want = dys.clone()
    dys.fill_(-5.0)
    assert sk.skinny_expert_combine_grad(dy.data_ptr(), dy.stride(0), 0, 0, T * k, pt.data_ptr(), wt.data_ptr(), k, T, k, H,
                                         sk.SKINNY_BF16 if dtype == "bf16" else sk.SKINNY_F32, dys.data_ptr(), ld, 0, 0,
                                         torch.cuda.current_stream().cuda_stream) == sk.SKINNY_OK
    assert torch.equal(dys, want)


@pytest.mark.parametrize("H,dtype", [(2047, "bf16"), (1, "bf16"), (9, "bf16"), (1018, "bf16"), (509, "fp32"), (1, "fp32"), (1027, "fp32")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (5, 3)])
def test_dispatch_copies_bits_at_any_alignment(H, dtype, pad, offset):
    """Every pattern of bits, NaN of any payload too, arrives as it is; the gaps between rows stay."""
    T, k, E = 700, 5, 37
    ids, _ = ref.routing(T, k, E, seed=H, drop=0.2)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    ld = H + pad
    g = torch.Generator().manual_seed(H)
    lo, hi = torch.iinfo(bits).min, torch.iinfo(bits).max
    x = torch.as_strided(torch.randint(lo, hi, (T * ld + offset + 8,), generator=g, dtype=bits).cuda().view(DT[dtype]), (T, H),
                         (ld, 1), offset)
    buf = torch.full((T * k * ld + offset + 16,), 77, dtype=bits, device="cuda")
    xs = torch.as_strided(buf.view(DT[dtype]), (T * k, H), (ld, 1), offset + 1)
    _, pos, order, off = sk.expert_dispatch(torch.from_numpy(ids).cuda(), E, x=x, xs=xs)
    rpos, rorder, roff = ref.dispatch(ids, E)
    n = int(roff[-1])
    assert np.array_equal(pos.cpu().numpy(), rpos)
    assert torch.equal(xs.view(bits)[:n], x.view(bits)[torch.from_numpy(rorder[:n].astype(np.int64)).cuda() // k])
    xs.view(bits)[:n] = 77
    assert (buf == 77).all()


def test_spread_bounded_wait_reports_and_recovers():
    T, k, H = 640, 4, 1001                    # more entries than one launch sorts
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda").reshape(T, k)
    ids, _ = ref.routing(T, k, 16, seed=1)
    it = torch.from_numpy(ids).cuda()
    for dtype in ("bf16", "fp32"):
        x, ys = matrix(T, H, dtype, 1), matrix(T * k, H, dtype, 2)
        for call in (lambda: sk.expert_dispatch(it, 16, x=x)[0], lambda: sk.expert_combine_grad(x, ys, pos)[0]):
            want = call()
            with sk.options(wait_timeout_us=0):
                call()
                torch.cuda.synchronize()
            assert sk.skinny_get_device_status() & 0xFF == sk.SKINNY_ERR_DEVICE_TIMEOUT
            for _ in range(2):
                assert torch.equal(call(), want)
            assert sk.skinny_get_device_status() == 0
