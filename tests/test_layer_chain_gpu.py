"""A dense layer's operators one behind the other, forward and backward, as a
training step and a decode step run them: each may start while the one before
it still runs.  Every result is checked against 64 bits from what the GPU's own
operators in front of it gave."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk
import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _init():
    assert sk.skinny_init(0) == sk.SKINNY_OK
    yield
    assert sk.skinny_get_device_status() == 0


class Layer:
    def __init__(self, T, Hq, Hk, D, hidden, inner, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.T, self.Hq, self.Hk, self.D, self.hidden, self.inner = g, T, Hq, Hk, D, hidden, inner

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        def buf(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        heads = Hq + 2 * Hk
        self.wqkv, self.bqkv, self.wo = weight(heads * D, hidden), weight(heads * D), weight(hidden, Hq * D)
        self.wgu, self.wd = weight(2 * inner, hidden), weight(hidden, inner)
        self.qw, self.kw = 1 + weight(D), 1 + weight(D)
        angle = torch.arange(300, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        self.table = torch.cat([angle.cos(), angle.sin()], dim=1).float().cuda()
        self.x, self.dy = buf(T, hidden), buf(T, hidden)
        self.positions = buf(T, dtype=torch.int32)
        self.qkv, self.q, self.k = buf(T, heads, D), buf(T, Hq, D), buf(T, Hk, D)
        self.h, self.act, self.pre, self.y = buf(T, hidden), buf(T, inner), buf(T, 2 * inner), buf(T, hidden)
        self.dact, self.dwd, self.dh, self.dwgu = buf(T, inner), buf(hidden, inner), buf(T, hidden), buf(2 * inner, hidden)
        self.dbgu = buf(2 * inner, dtype=torch.float32)
        self.do, self.dwo = buf(T, Hq * D), buf(hidden, Hq * D)
        self.dq, self.dk, self.dqw, self.dkw = buf(T, Hq, D), buf(T, Hk, D), buf(D, dtype=torch.float32), buf(D, dtype=torch.float32)
        self.outs = [self.qkv, self.q, self.k, self.h, self.act, self.pre, self.y, self.dact, self.dwd, self.dh, self.dwgu, self.dbgu,
                     self.do, self.dwo, self.dq, self.dk, self.dqw, self.dkw]
        need = max(sk.linear_grad_workspace(self.dy, self.act, self.wd),
                   sk.linear_grad_workspace(self.dact, self.h, self.wgu, "swiglu"),
                   sk.linear_grad_workspace(self.dh, self.q.view(T, -1), self.wo),
                   sk.linear_workspace(self.x, self.wqkv), sk.linear_workspace(self.q.view(T, -1), self.wo),
                   sk.linear_workspace(self.h, self.wgu, "swiglu"), sk.linear_workspace(self.act, self.wd),
                   sk.qk_norm_rope_grad_workspace(T, Hq, Hk, D))
        self.space = buf(need, dtype=torch.uint8)      # one for all: the calls follow each other on a stream

    def views(self):
        return self.qkv[:, :self.Hq], self.qkv[:, self.Hq:self.Hq + self.Hk]

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x.copy_(torch.randn((self.T, self.hidden), generator=g, device="cuda"))
        self.dy.copy_(torch.randn((self.T, self.hidden), generator=g, device="cuda"))
        self.positions.copy_(torch.randint(0, 300, (self.T,), generator=g, device="cuda"))

    def step(self, train=True):
        ws = dict(workspace=self.space)
        sk.linear(self.x, self.wqkv, bias=self.bqkv, out=self.qkv.view(self.T, -1), **ws)
        q, k = self.views()
        sk.qk_norm_rope(q, k, self.qw, self.kw, self.table, self.positions, q_out=self.q, k_out=self.k)
        sk.linear(self.q.view(self.T, -1), self.wo, residual=self.x, out=self.h, **ws)
        sk.linear(self.h, self.wgu, activation="swiglu", out=self.act, pre=self.pre if train else None, **ws)
        sk.linear(self.act, self.wd, residual=self.h, out=self.y, **ws)
        if not train:
            return
        sk.linear_grad(self.dy, self.act, self.wd, dx=self.dact, dw=self.dwd, **ws)
        sk.linear_grad(self.dact, self.h, self.wgu, pre=self.pre, activation="swiglu", dx=self.dh, dw=self.dwgu, dbias=self.dbgu,
                       bias_grad=True, **ws)
        sk.linear_grad(self.dh, self.q.view(self.T, -1), self.wo, dx=self.do, dw=self.dwo, **ws)
        sk.qk_norm_rope_grad(self.do.view(self.T, self.Hq, self.D), self.k, q, k, self.qw, self.kw, self.table, self.positions,
                             dq_in=self.dq, dk_in=self.dk, dq_weight=self.dqw, dk_weight=self.dkw, **ws)

    def check(self, train=True):
        T, bf = self.T, torch.bfloat16

        def product(got, x, w, b=None, act=None, r=None, pre=None):
            y, z, size = ref.linear(x, w, b, act, r)
            ref.check(got, y, ref.linear_bound(y, z, size, act, r, bf))

        product(self.qkv.view(T, -1), self.x, self.wqkv, self.bqkv)
        cos, sin = ref.angles(self.table, self.positions, None, T)
        for src, w, got in zip(self.views(), (self.qw, self.kw), (self.q, self.k)):
            ref.check(got, *ref.heads(src, w, cos, sin, 1e-6, False, bf))
        product(self.h, self.q.view(T, -1), self.wo, r=self.x)
        product(self.act, self.h, self.wgu, act="swiglu")
        product(self.y, self.act, self.wd, r=self.h)
        if not train:
            return
        for dy, x, w, z, act, got in ((self.dy, self.act, self.wd, None, None, (self.dact, self.dwd)),
                                      (self.dact, self.h, self.wgu, self.pre, "swiglu", (self.dh, self.dwgu, self.dbgu)),
                                      (self.dh, self.q.view(T, -1), self.wo, None, None, (self.do, self.dwo))):
            for t, (want, bound) in zip(got, ref.linear_grad(dy, x, w, z, act)):
                ref.check(t, want, bound)
        q, k = self.views()
        for d, src, w, dx, dw in ((self.do.view(T, self.Hq, self.D), q, self.qw, self.dq, self.dqw), (self.k, k, self.kw, self.dk, self.dkw)):
            (want, bound), (wsum, wbound) = ref.heads_grad(d, src, w, cos, sin, 1e-6, False, bf)
            ref.check(dx, want, bound)
            ref.check(dw, wsum, wbound)


SIZES = [(1, 8, 2, 64, 512, 264), (16, 4, 1, 128, 768, 1024), (61, 7, 1, 72, 520, 328), (300, 8, 2, 64, 640, 512),
         (13, 3, 3, 10, 51, 33), (700, 4, 4, 64, 256, 1000)]


@pytest.mark.parametrize("pdl", [0, 1, 2])
@pytest.mark.parametrize("size", SIZES)
def test_step(size, pdl):
    with sk.options(pdl=pdl):
        layer = Layer(*size)
        layer.fill(1)
        layer.step()
        layer.check()


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("size", SIZES[:4])
def test_captured_steps_on_new_inputs(size, train):
    with sk.options(pdl=1):
        layer = Layer(*size)
        layer.fill(1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.step(train)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.step(train)
        for seed in (2, 3):
            layer.fill(seed)
            layer.step(train)
            eager = [t.clone() for t in layer.outs]
            for t in layer.outs:
                t.fill_(float("nan"))
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            used = range(len(eager)) if train else (0, 1, 2, 3, 4, 6)
            assert all(torch.equal(layer.outs[i], eager[i]) for i in used)
        layer.check(train)


def test_two_layers_at_once():
    """Two streams, each with buffers and a workspace of its own."""
    layers = [Layer(*SIZES[3], seed=s) for s in (0, 1)]
    for s, layer in enumerate(layers):
        layer.fill(s)
        layer.step()
    alone = [[t.clone() for t in layer.outs] for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for layer in layers:
        for t in layer.outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                layer.step()
    torch.cuda.synchronize()
    for layer, want in zip(layers, alone):
        assert all(torch.equal(a, b) for a, b in zip(layer.outs, want))


@pytest.mark.parametrize("backend", [sk.SKINNY_BACKEND_TCGEN05, sk.SKINNY_BACKEND_SPLITK])
@pytest.mark.parametrize("M,act", [(5, None), (300, "swiglu"), (2000, None)])
def test_a_wait_that_gives_up_reports_and_later_calls_work(M, act, backend):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, 1024), generator=g, device="cuda").bfloat16()
    w = torch.randn((512, 1024), generator=g, device="cuda").bfloat16()
    with sk.options(backend=backend):
        want = sk.linear(x, w, activation=act)
        torch.cuda.synchronize()
        with sk.options(wait_timeout_us=0):
            sk.linear(x, w, activation=act)
            torch.cuda.synchronize()
        assert sk.skinny_get_device_status() & 0xFF == sk.SKINNY_ERR_DEVICE_TIMEOUT
        assert torch.equal(sk.linear(x, w, activation=act), want)
    assert sk.skinny_get_device_status() == 0


@pytest.mark.parametrize("pdl", [1, 2])
def test_beside_the_other_kernels_with_tensor_memory(pdl):
    """The projections, the experts' products and these products by turns, each allowed to start while the one
    before it still runs: all of them take tensor memory, and none waits for another's."""
    g = torch.Generator(device="cuda").manual_seed(4)

    def rand(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 0.1).bfloat16()

    x, big, w, we = rand(40, 1024), rand(1300, 1024), rand(2112, 1024), rand(8, 512, 1024)
    offsets = torch.tensor([0, 5, 10, 15, 20, 25, 30, 35, 40], dtype=torch.int32, device="cuda")
    q = rand(40, 8, 128)

    def steps():
        out = []
        for i in range(12):
            with sk.options(backend=sk.SKINNY_BACKEND_TCGEN05):
                out.append(sk.gemm(x, w))
                out.append(sk.experts_gemm(x, offsets, we))
                out.append(sk.linear(big[:100 + 100 * i], w, activation="silu"))
            with sk.options(backend=sk.SKINNY_BACKEND_SPLITK):
                out.append(sk.linear(x[:1 + 3 * i], w, activation="swiglu"))
                out.append(sk.linear(big[:90], w[:128 + 8 * i]))
            out.append(sk.qk_norm_rope(q, None)[0])
            out.extend(sk.linear_grad(out[-3][:, :1056], x[:1 + 3 * i], w, activation="swiglu",
                                      pre=out[-4][:1 + 3 * i])[:2])
        return out

    want = [t.clone() for t in steps()]
    torch.cuda.synchronize()
    with sk.options(pdl=pdl):
        for _ in range(3):
            got = steps()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("between", [False, True])
@pytest.mark.parametrize("M,N,K,act", [(1, 2112, 4096, None), (64, 1024, 1024, "swiglu"), (5, 300, 201, "gelu"),
                                       (600, 2048, 2048, None)])
@pytest.mark.parametrize("pdl", [1, 2])
def test_weights_that_a_call_just_before_writes(M, N, K, act, between, pdl):
    """In the stream's order, whatever starts early: as with a wait between any two calls."""
    rows = 2 * N if act == "swiglu" else N
    g = torch.Generator(device="cuda").manual_seed(M)

    def new(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, device="cuda", dtype=dtype)

    lefts, right, few, x, z = [new(rows, 64) for _ in range(6)], new(K, 64), new(64, K), new(M, K), new(M, rows)
    w, other, dy = buf(rows, K), buf(M, 64), new(M, N)
    outs, grads = [buf(M, N) for _ in lefts], [buf(M, K) for _ in lefts]
    space = buf(sk.linear_grad_workspace(dy, x, w, act), dtype=torch.uint8)

    def run(wait):
        w.zero_()
        wait()
        for left, out, dx in zip(lefts, outs, grads):
            sk.linear(left, right, out=w)
            if between:
                wait()
                sk.linear(x, few, out=other)
            wait()
            sk.linear(x, w, activation=act, out=out)
            wait()
            sk.linear_grad(dy, x, w, z if act else None, act, dx=dx, weight_grad=False, workspace=space)
            wait()
        torch.cuda.synchronize()
        return [t.clone() for t in outs + grads]

    with sk.options(pdl=pdl):
        want = run(torch.cuda.synchronize)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))


@pytest.mark.parametrize("M,N,K,act", [(33, 513, 511, "gelu"), (64, 256, 512, "swiglu"), (700, 640, 1000, None),
                                       (2000, 1437, 520, "silu"), (1, 130, 70, None), (300, 77, 2048, "geglu")])
def test_gradients_one_behind_another_in_one_workspace(M, N, K, act):
    """Any choice of outputs, each call on the workspace of the one before: the same with launches that overlap."""
    rows = 2 * N if act in ("swiglu", "geglu") else N
    g = torch.Generator(device="cuda").manual_seed(N)

    def new(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    sets = [(new(M, N), new(M, K), new(rows, K), new(M, rows)) for _ in range(3)]
    choices = [(dx, dw, db) for dx in (0, 1) for dw in (0, 1) for db in (0, 1) if dx or dw or db]
    space = torch.empty(sk.linear_grad_workspace(*sets[0][:3], act), device="cuda", dtype=torch.uint8)
    outs = [(torch.empty(M, K, device="cuda", dtype=torch.bfloat16), torch.empty(rows, K, device="cuda", dtype=torch.bfloat16),
             torch.empty(rows, device="cuda")) for _ in range(2 * len(choices))]

    def run(pdl):
        for out in outs:
            for t in out:
                t.fill_(-7)
        with sk.options(pdl=pdl):
            for i, out in enumerate(outs):
                dx, dw, db = choices[i * 3 % len(choices)]
                dy, x, w, z = sets[i % 3]
                sk.linear_grad(dy, x, w, z if act else None, act, dx=out[0] if dx else None, dw=out[1] if dw else None,
                               dbias=out[2] if db else None, input_grad=dx, weight_grad=dw, bias_grad=db, workspace=space)
        torch.cuda.synchronize()
        return [t.clone() for out in outs for t in out]

    want = run(0)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(run(1), want))
