"""Products with bias, activation and residual, and their gradients, against 64 bits."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk
import layer_ref as ref

pytestmark = pytest.mark.gpu

CANARY = -7777.0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def strided(t, ld, offset=0):
    """The same rows, `ld` apart, `offset` elements into a buffer."""
    m, n = t.shape
    buf = torch.full((offset + m * ld + 8,), CANARY, dtype=t.dtype, device=t.device)
    view = buf[offset:offset + m * ld].view(m, ld)[:, :n]
    view.copy_(t)
    return view


def gaps_kept(view):
    """What lies around a strided output is as it was."""
    buf = view._base if view._base is not None else view
    buf = buf.clone().view(-1)
    m, n = view.shape
    off = view.storage_offset()
    torch.as_strided(buf, (m, n), view.stride(), off).fill_(CANARY)
    return bool((buf == torch.tensor(CANARY, dtype=buf.dtype)).all())


def forward(M, N, K, act, bias=True, residual=True, out=torch.bfloat16, pre=True, seed=0, pad=(0, 0, 0), offset=(0, 0, 0)):
    g = gen(seed)
    rows = 2 * N if act in ref.GATED else N
    x = strided(rand(g, M, K), K + pad[0], offset[0])
    w = strided(rand(g, rows, K, scale=K ** -0.5 if K else 1.0), K + pad[1], offset[1])
    b = rand(g, rows, scale=0.5) if bias else None
    r = strided(rand(g, M, N, dtype=out), N + 3) if residual else None
    y = strided(torch.full((M, N), CANARY, dtype=out, device="cuda"), N + pad[2], offset[2])
    z = strided(torch.full((M, rows), CANARY, dtype=torch.bfloat16, device="cuda"), rows + pad[2], offset[2]) if pre else None
    got = sk.linear(x, w, bias=b, activation=act, residual=r, out=y, pre=z)
    assert got is y
    want, zz, size = ref.linear(x, w, b, act, r)
    ref.check(y, want, ref.linear_bound(want, zz, size, act, r, out), "y")
    assert gaps_kept(y)
    if pre:
        dz = 1e-5 * size + 1e-6
        ref.check(z, zz, dz + 2.0 ** -8 * 1.01 * (zz.abs() + dz), "pre")
        assert gaps_kept(z)
    return x, w, b, r, y, z


ACTS = [None, "silu", "gelu", "swiglu", "geglu"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (1, 2112, 512), (2, 80, 7168), (5, 200, 136), (16, 256, 1024), (17, 96, 264),
                                   (64, 320, 512), (61, 136, 2048), (65, 72, 128), (200, 264, 320), (300, 1024, 72)])
def test_linear(M, N, K, act):
    forward(M, N, K, act)


@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 7, 9), (3, 33, 65), (16, 61, 1000), (31, 129, 257), (64, 65, 63),
                                   (100, 127, 129), (259, 130, 515), (1, 1000, 7)])
def test_odd_sizes(M, N, K, act):
    forward(M, N, K, act)
    forward(M, N, K, act, out=torch.float32, pre=False)


@pytest.mark.parametrize("M", [1, 9, 40, 130])
@pytest.mark.parametrize("pad,offset", [((8, 16, 24), (0, 0, 0)), ((1, 0, 1), (0, 0, 0)), ((0, 3, 5), (1, 0, 1)),
                                        ((8, 8, 8), (4, 8, 3)), ((2, 4, 2), (8, 1, 2))])
def test_strides_and_alignment(M, pad, offset):
    for act in (None, "swiglu"):
        forward(M, 168, 320, act, pad=pad, offset=offset, seed=M)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [4, 33, 150])
def test_parts_of_the_epilogue(M, out, residual, bias):
    for act in (None, "silu", "geglu"):
        forward(M, 144, 256, act, bias=bias, residual=residual, out=out, pre=False)


@pytest.mark.parametrize("M,N,K", [(1024, 512, 512), (1000, 768, 320), (2047, 520, 1160), (129, 4096, 256), (513, 2112, 192),
                                   (3000, 256, 64)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_many_rows(M, N, K, act):
    forward(M, N, K, act)


@pytest.mark.parametrize("M", [2, 64, 300])
def test_residual_in_place(M):
    g = gen(5)
    x, w, y = rand(g, M, 256), rand(g, 136, 256, scale=1 / 16), rand(g, M, 136)
    r = y.clone()
    assert sk.linear(x, w, residual=y, out=y) is y
    assert torch.equal(y, sk.linear(x, w, residual=r))


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("M", [3, 70, 600])
def test_residual_in_place_activated(M, act):
    g = gen(15)
    x, w, y = rand(g, M, 264), rand(g, 2 * 136, 264, scale=1 / 16), rand(g, M, 136 if act == "swiglu" else 272, dtype=torch.float32)
    want = sk.linear(x, w, activation=act, residual=y.clone())
    assert want.dtype == torch.float32
    assert torch.equal(sk.linear(x, w, activation=act, residual=y, out=y), want)


@pytest.mark.parametrize("ld", [(1 << 30) + 8, (1 << 30) + 3])
def test_rows_past_32_bits(ld):
    """Row strides that carry the last rows past 2^32 bytes, of every operand and output."""
    g = gen(16)
    M, N, K = 4, 3, 136
    x, w, dy = rand(g, M, K), rand(g, N, K), rand(g, M, N)
    want, dwant = sk.linear(x, w), sk.linear_grad(dy, x, w, bias_grad=True)
    bufs = [torch.empty(3 * ld + 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far = torch.as_strided(bufs[0], (M, K), (ld, 1))
    far.copy_(x)
    out = torch.as_strided(bufs[1], (M, N), (ld, 1))
    assert torch.equal(sk.linear(far, w, out=out), want)
    dx = torch.as_strided(bufs[1], (M, K), (ld, 1))
    got = sk.linear_grad(dy, far, w, dx=dx, bias_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(got, dwant))
    wide = torch.as_strided(bufs[0], (N, K), (ld, 1))
    wide.copy_(w)
    dw = torch.as_strided(bufs[1], (N, K), (ld, 1))
    got = sk.linear_grad(dy, x, wide, dw=dw, bias_grad=True)
    assert torch.equal(sk.linear(x, wide), want) and all(torch.equal(a, b) for a, b in zip(got, dwant))


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_very_many_rows(act):
    forward(200003, 40, 64, act)
    backward(70001, 40, 72, act)


@pytest.mark.parametrize("M", [1, 40, 100])
def test_same_sign_sums(M):
    """Nothing cancels: a biased sum would show."""
    g = gen(6)
    x = rand(g, M, 14336).abs()
    w = rand(g, 64, 14336).abs()
    y = torch.empty((M, 64), dtype=torch.float32, device="cuda")
    sk.linear(x, w, out=y)
    want, _, size = ref.linear(x, w, None, None, None)
    ref.check(y, want, 1e-5 * size, "same sign")


@pytest.mark.parametrize("M", [1, 20, 80])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
def test_far_values(M, act):
    """Activations far out on both sides are finite, zero or the identity."""
    N = 64
    rows = 2 * N if act in ref.GATED else N
    x = torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    w = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([-3e4, -200.0, -89.0, -30.0, -10.0, -1.0, 0.0, 1.0, 10.0, 89.0, 200.0, 3e4], device="cuda")
    w[:N, 0] = far.repeat(6)[:N].bfloat16()
    w[N:, 0] = 2
    y = torch.empty((M, N), dtype=torch.float32, device="cuda")
    sk.linear(x, w, activation=act, out=y)
    want, z, size = ref.linear(x, w, None, act, None)
    assert torch.isfinite(y).all()
    ref.check(y, want, ref.linear_bound(want, z, size, act, None, torch.float32), act)


@pytest.mark.parametrize("M", [3, 70])
def test_nan_and_infinity_stay_in_their_row(M):
    g = gen(7)
    x, w = rand(g, M, 128), rand(g, 96, 128, scale=0.1)
    clean = sk.linear(x, w)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y = sk.linear(x, w)
    assert y[1].isnan().all() and not torch.isfinite(y[2]).any()
    rest = [m for m in range(M) if m not in (1, 2)]
    assert torch.equal(y[rest], clean[rest])


def test_empty():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    w, b, r = torch.zeros((24, 0), **bf), torch.randn(24, device="cuda").bfloat16(), torch.randn((5, 24), device="cuda").bfloat16()
    y = sk.linear(torch.zeros((5, 0), **bf), w, bias=b, activation="gelu", residual=r)      # the empty sum
    want, z, size = ref.linear(torch.zeros((5, 0)), torch.zeros((24, 0)), b, "gelu", r)
    ref.check(y, want, ref.linear_bound(want, z, size, "gelu", r, torch.bfloat16), "K 0")
    for M in (40, 100):
        y = sk.linear(torch.zeros((M, 0), **bf), torch.zeros((24, 0), **bf), bias=b, activation="swiglu")
        want, z, size = ref.linear(torch.zeros((M, 0)), torch.zeros((24, 0)), b, "swiglu", None)
        ref.check(y, want, ref.linear_bound(want, z, size, "swiglu", None, torch.bfloat16), "K 0, gated")
    assert sk.linear(torch.zeros((0, 16), **bf), torch.zeros((8, 16), **bf)).shape == (0, 8)
    assert sk.linear(torch.zeros((4, 16), **bf), torch.zeros((0, 16), **bf)).shape == (4, 0)
    dx, dw, db = sk.linear_grad(torch.zeros((0, 8), **bf), torch.zeros((0, 16), **bf), torch.ones((8, 16), **bf), bias_grad=True)
    assert dx.shape == (0, 16) and not dw.any() and not db.any() and dw.shape == (8, 16)
    dx, dw, db = sk.linear_grad(torch.zeros((4, 0), **bf), torch.zeros((4, 16), **bf), torch.ones((0, 16), **bf), bias_grad=True)
    assert not dx.any() and dx.shape == (4, 16) and dw.shape == (0, 16)
    dx, dw, db = sk.linear_grad(torch.ones((4, 8), **bf), torch.zeros((4, 0), **bf), torch.ones((8, 0), **bf), bias_grad=True)
    assert torch.equal(db, torch.full((8,), 4.0, device="cuda"))


# ------------------------------------------------------------------ gradients

def backward(M, N, K, act, bias=True, seed=0, pad=0, offset=0):
    g = gen(seed)
    rows = 2 * N if act in ref.GATED else N
    dy = strided(rand(g, M, N), N + pad, offset)
    x = strided(rand(g, M, K), K + pad, offset)
    w = strided(rand(g, rows, K, scale=K ** -0.5), K + pad, offset)
    z = strided(rand(g, M, rows, scale=2.0), rows + pad, offset) if act else None
    dx = strided(torch.full((M, K), CANARY, dtype=torch.bfloat16, device="cuda"), K + 2 * pad, offset)
    dw = strided(torch.full((rows, K), CANARY, dtype=torch.bfloat16, device="cuda"), K + pad, offset)
    out = sk.linear_grad(dy, x, w, pre=z, activation=act, dx=dx, dw=dw, bias_grad=bias)
    assert out[0] is dx and out[1] is dw and (out[2] is not None) == bias
    for name, got, (want, bound) in zip(("dx", "dw", "dbias"), out, ref.linear_grad(dy, x, w, z, act)):
        if got is not None:
            ref.check(got, want, bound, name)
    assert gaps_kept(dx) and gaps_kept(dw)
    return dy, x, w, z, out


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (7, 136, 72), (64, 256, 320), (130, 200, 264), (515, 512, 192)])
def test_grad(M, N, K, act):
    backward(M, N, K, act)


@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 7), (33, 61, 127), (129, 131, 65), (1001, 67, 130), (2, 1437, 50)])
def test_grad_odd_sizes(M, N, K, act):
    backward(M, N, K, act)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (4, 8), (8, 1), (0, 3)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_grad_strides(pad, offset, act):
    backward(70, 136, 200, act, pad=pad, offset=offset)


@pytest.mark.parametrize("M,N,K", [(2048, 512, 768), (1000, 1024, 2048), (64, 2048, 1024), (4096, 72, 320), (300, 4096, 136)])
def test_grad_many(M, N, K):
    backward(M, N, K, None, bias=False)
    backward(M, N, K, "swiglu")


def test_grad_parts():
    """Each gradient by itself is what all of them together give."""
    dy, x, w, z, (dx, dw, db) = backward(100, 136, 264, "geglu")
    kw = dict(pre=z, activation="geglu")
    assert torch.equal(sk.linear_grad(dy, x, w, weight_grad=False, **kw)[0], dx)
    assert torch.equal(sk.linear_grad(dy, x, w, input_grad=False, **kw)[1], dw)
    only = sk.linear_grad(dy, x, w, input_grad=False, weight_grad=False, bias_grad=True, **kw)
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
def test_gradient_against_differences(act):
    """Along a direction of Z, with the loss <dy, y> in 64 bits: central differences of the definition against
    what the kernel's dbias says (a shift of the bias is a shift of Z)."""
    g = gen(9)
    M, N, K = 37, 24, 40
    rows = 2 * N if act in ref.GATED else N
    x, w, b = rand(g, M, K), rand(g, rows, K, scale=0.3), rand(g, rows)
    z = torch.empty((M, rows), dtype=torch.bfloat16, device="cuda")
    sk.linear(x, w, bias=b, activation=act, pre=z)
    dy = rand(g, M, N)
    db = sk.linear_grad(dy, x, w, pre=z, activation=act, input_grad=False, weight_grad=False, bias_grad=True)[2]

    def loss(zz):
        y = ref.act_both(act, zz[:, :N])[0]
        return ((y * zz[:, N:] if act in ref.GATED else y) * dy.double().cpu()).sum().item()

    h = 1e-5
    for j in range(0, rows, 5):
        e = torch.zeros(rows, dtype=torch.double)
        e[j] = h
        diff = (loss(z.double().cpu() + e) - loss(z.double().cpu() - e)) / (2 * h)
        assert abs(diff - db[j].item()) <= 1e-4 * (1 + dy.double().abs().sum().item() * 0.01)


@pytest.mark.parametrize("act", ["gelu", "geglu", "silu"])
def test_grad_far_values(act):
    """Kept sums up to the largest bf16 values have finite gradients."""
    N = 16
    rows = 2 * N if act in ref.GATED else N
    far = torch.tensor([-3e38, -1e20, -1e13, -500.0, -88.0, -5.0, 0.0, 5.0, 88.0, 500.0, 1e13, 1e20, 3e38, 1.0, -1.0, 0.5])
    z = torch.ones((4, rows), dtype=torch.bfloat16, device="cuda")
    z[:, :N] = far.bfloat16().cuda()
    dy = torch.ones((4, N), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((4, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((rows, 8), dtype=torch.bfloat16, device="cuda")
    db = sk.linear_grad(dy, x, w, pre=z, activation=act, bias_grad=True)[2].cpu()[:N]
    assert torch.isfinite(db).all()
    want = torch.where(far > 80, 4.0, 0.0)
    at = (far.abs() > 80)
    assert torch.allclose(db[at], want[at], atol=1e-30)


# ------------------------------------------------------------------ each kernel

KERNELS = {"pair": sk.SKINNY_BACKEND_TCGEN05, "split": sk.SKINNY_BACKEND_SPLITK}


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (130, 72, 64), (256, 256, 256), (257, 264, 320), (600, 520, 1096), (1, 700, 4104),
                                   (2305, 136, 72)])
def test_kernels_agree_with_64_bits(M, N, K, act, kernel):
    with sk.options(backend=KERNELS[kernel]):
        forward(M, N, K, act)
        forward(M, N, K, act, out=torch.float32, bias=False, residual=False, pre=False)
        backward(M, N, K, act)


@pytest.mark.parametrize("act", [None, "geglu"])
def test_pair_walks_many_tiles(act):
    """More tiles than pairs of SMs, the last band of rows short."""
    with sk.options(backend=sk.SKINNY_BACKEND_TCGEN05):
        forward(2700, 2312, 200, act)
        backward(2700, 2312, 328, act)


@pytest.mark.parametrize("kernel", ["pair", "split"])
def test_same_sign_sums_each_kernel(kernel):
    g = gen(6)
    for M in (16, 300):
        x, w = rand(g, M, 14336).abs(), rand(g, 256, 14336).abs()
        y = torch.empty((M, 256), dtype=torch.float32, device="cuda")
        with sk.options(backend=KERNELS[kernel]):
            sk.linear(x, w, out=y)
        want, _, size = ref.linear(x, w, None, None, None)
        ref.check(y, want, 1e-5 * size, kernel)


# ------------------------------------------------------------------ calls

def calls(M):
    g = gen(M)
    x, w = rand(g, M, 512), rand(g, 2 * 264, 512, scale=1 / 16)
    y, z = torch.empty((M, 264), dtype=torch.bfloat16, device="cuda"), torch.empty((M, 528), dtype=torch.bfloat16, device="cuda")
    dy = rand(g, M, 264)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(528, device="cuda")
    space = torch.empty(sk.linear_grad_workspace(dy, x, w, "swiglu"), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        sk.linear(x, w, activation="swiglu", out=y, pre=z, stream=stream)
        sk.linear_grad(dy, x, w, pre=z, activation="swiglu", dx=dx, dw=dw, dbias=db, bias_grad=True, workspace=space,
                       stream=stream)
        return [y, z, dx, dw, db]
    return step


@pytest.mark.parametrize("pdl", [0, 1])
@pytest.mark.parametrize("M", [1, 24, 200, 700])
def test_same_bits_again_captured_and_on_a_stream(M, pdl):
    with sk.options(pdl=pdl):
        step = calls(M)
        first = [t.clone() for t in step()]
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, step()))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(first, out))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for t in out:
            t.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    assert sk.skinny_get_device_status() == 0


def test_tensor_functions_refuse():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w = torch.zeros((4, 16), **bf), torch.zeros((8, 16), **bf)
    with pytest.raises(ValueError):
        sk.linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        sk.linear(x, torch.zeros((7, 16), **bf), activation="swiglu")
    with pytest.raises(ValueError):
        sk.linear(x, torch.zeros((8, 15), **bf))
    with pytest.raises(TypeError):
        sk.linear(x.float(), w)
    with pytest.raises(TypeError):
        sk.linear(x, w, bias=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        sk.linear(x, w, bias=torch.zeros(9, **bf))
    with pytest.raises(TypeError):
        sk.linear(x, w, residual=torch.zeros((4, 8), device="cuda"), out=torch.zeros((4, 8), **bf))
    with pytest.raises(ValueError):
        sk.linear(x, w, pre=torch.zeros((4, 9), **bf))
    with pytest.raises(sk.SkinnyError):
        sk.linear(x, w, out=x[:, :8])
    with pytest.raises(ValueError):
        sk.linear_grad(torch.zeros((4, 8), **bf), x, w, activation="silu")
    with pytest.raises(ValueError):
        sk.linear_grad(torch.zeros((4, 8), **bf), x, w, dx=x, input_grad=False)
    with pytest.raises(sk.SkinnyError):
        sk.linear_grad(torch.zeros((4, 8), **bf), x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
