"""Norms of queries and keys with the position rotation, and their gradients, against 64 bits."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk
import layer_ref as ref

pytestmark = pytest.mark.gpu

CANARY = -7777.0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def table(P, R, theta=1e4):
    angle = torch.arange(P, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().cuda()


class Case:
    def __init__(self, T, Hq, Hk, D, R=None, axes=1, interleaved=False, eps=1e-6, dtype=torch.bfloat16, weights=True, seed=0,
                 layout="fused", P=500):
        g = gen(seed)
        self.T, self.D, self.eps, self.dtype, self.interleaved = T, D, eps, dtype, interleaved
        R = D // 2 * 2 if R is None else R
        if layout == "fused":               # beside the values, in the projection's rows
            rows = torch.randn((T, Hq + 2 * Hk, D), generator=g, device="cuda").to(dtype)
            self.q, self.k = rows[:, :Hq], rows[:, Hq:Hq + Hk]
        elif layout == "heads first":
            self.q = torch.randn((Hq, T, D), generator=g, device="cuda").to(dtype).transpose(0, 1)
            self.k = torch.randn((Hk, T, D), generator=g, device="cuda").to(dtype).transpose(0, 1)
        else:                               # rows that lie on no boundary
            self.q = torch.randn((T, Hq, D + 3), generator=g, device="cuda").to(dtype)[..., 1:D + 1]
            self.k = torch.randn((T, Hk, D + 1), generator=g, device="cuda").to(dtype)[..., :D]
        w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
        self.qw, self.kw = w if weights and eps is not None else (None, None)
        self.table = table(P, R) if R else None
        self.positions = torch.randint(0, P, (axes, T), generator=g, device="cuda", dtype=torch.int32) if R else None
        self.pair_axis = (torch.randint(0, axes, (R // 2,), generator=g, device="cuda", dtype=torch.int32)
                          if axes > 1 and R else None)
        self.dq = torch.randn((T, Hq, D), generator=g, device="cuda").to(dtype)
        self.dk = torch.randn((T, Hk, D), generator=g, device="cuda").to(dtype)

    def angles(self):
        return ref.angles(self.table, self.positions, self.pair_axis, self.T) if self.table is not None else (None, None)

    def kw_args(self):
        return dict(q_weight=self.qw, k_weight=self.kw, table=self.table, positions=self.positions, eps=self.eps,
                    pair_axis=self.pair_axis, interleaved=self.interleaved)

    def run(self, **kw):
        return sk.qk_norm_rope(self.q, self.k, **self.kw_args(), **kw)

    def grad(self, **kw):
        return sk.qk_norm_rope_grad(self.dq, self.dk, self.q, self.k, **self.kw_args(), **kw)

    def check(self, outs=None):
        cos, sin = self.angles()
        outs = outs or self.run()
        for name, x, w, y in (("q", self.q, self.qw, outs[0]), ("k", self.k, self.kw, outs[1])):
            want, bound = ref.heads(x, w, cos, sin, self.eps, self.interleaved, self.dtype)
            ref.check(y, want, bound, name)
        return outs

    def check_grad(self, outs=None):
        cos, sin = self.angles()
        outs = outs or self.grad()
        for name, d, x, w, dx, dw in (("q", self.dq, self.q, self.qw, outs[0], outs[2]), ("k", self.dk, self.k, self.kw, outs[1], outs[3])):
            (want, bound), weight = ref.heads_grad(d, x, w, cos, sin, self.eps, self.interleaved, self.dtype)
            ref.check(dx, want, bound, "d" + name)
            if weight is None:
                assert dw is None
            else:
                ref.check(dw, weight[0], weight[1], f"d{name} weight")
        return outs


SIZES = [(1, 1, 1, 2), (1, 32, 8, 128), (3, 7, 1, 64), (64, 32, 8, 128), (200, 12, 12, 72), (5, 5, 3, 61), (17, 3, 2, 511),
         (9, 2, 2, 512), (33, 16, 2, 80), (2, 128, 1, 192), (1000, 4, 4, 96), (7, 1, 1, 1), (1500, 9, 3, 40)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,D", SIZES)
def test_heads(T, Hq, Hk, D, dtype):
    for interleaved in (False, True):
        c = Case(T, Hq, Hk, D, interleaved=interleaved, dtype=dtype)
        c.check()
        c.check_grad()


@pytest.mark.parametrize("layout", ["fused", "heads first", "unaligned"])
@pytest.mark.parametrize("axes", [1, 2, 3, 8])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (96, 36), (72, 36), (61, 60), (256, 0), (80, 2), (30, 10)])
def test_axes_parts_and_layouts(D, R, axes, layout):
    for interleaved in (False, True):
        for dtype in (torch.bfloat16, torch.float32):
            c = Case(21, 6, 3, D, R=R, axes=axes, layout=layout, interleaved=interleaved, dtype=dtype, seed=D + axes)
            c.check()
            c.check_grad()


@pytest.mark.parametrize("eps,weights", [(None, False), (1e-6, False), (0.5, True)])
def test_norm_and_weights(eps, weights):
    for D, R in ((128, 128), (80, 40)):
        c = Case(50, 8, 2, D, R=R, eps=eps, weights=weights)
        c.check()
        outs = c.check_grad()
        assert (outs[2] is None) == (eps is None)


def test_rotation_alone_is_exact_where_it_turns_nothing():
    c = Case(10, 4, 2, 64, eps=None)
    c.positions.fill_(-1)
    q, k = c.run()
    assert torch.equal(q, c.q) and torch.equal(k, c.k)


def test_positions_and_axes_outside():
    c = Case(40, 4, 2, 64, axes=2)
    c.positions[0, ::3] = -1
    c.positions[1, 1::3] = 500
    c.positions[0, 5] = 2 ** 31 - 1
    c.positions[1, 6] = -2 ** 31
    c.pair_axis[3] = 2
    c.pair_axis[4] = -1
    c.check()
    c.check_grad()


@pytest.mark.parametrize("layout", ["fused", "unaligned"])
def test_in_place(layout):
    c = Case(30, 6, 2, 64, layout=layout)
    want = [t.clone() for t in c.run()]
    dwant = [t.clone() for t in c.grad()]
    got = c.grad(dq_in=c.dq, dk_in=c.dk)
    assert all(torch.equal(a, b) for a, b in zip(dwant, got))
    q, k = c.run(q_out=c.q, k_out=c.k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_rest_of_the_rows_is_kept():
    T, D = 12, 64
    rows = torch.full((T, 10, D + 8), CANARY, device="cuda").bfloat16()
    c = Case(T, 5, 2, D)
    q, k = rows[:, 1:6, :D], rows[:, 7:9, :D]
    got = c.run(q_out=q, k_out=k)
    want = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q.fill_(CANARY)
    k.fill_(CANARY)
    assert (rows == torch.tensor(CANARY).bfloat16().item()).all()


def test_zero_rows_infinities_and_nan_stay_in_their_head():
    c = Case(8, 4, 2, 128)
    clean = c.run()[0]
    c.q[2, 1] = 0
    c.q[3, 2, 5] = float("nan")
    c.q[4, 0, 9] = float("inf")
    q = c.run()[0]
    assert not q[2, 1].any()                # eps keeps a row of zeros finite
    assert q[3, 2].isnan().all()
    assert q[4, 0].isnan().any()
    keep = torch.ones((8, 4), dtype=torch.bool)
    keep[2, 1] = keep[3, 2] = keep[4, 0] = False
    assert torch.equal(q[keep], clean[keep])


def test_one_kind_alone():
    c = Case(20, 5, 2, 64)
    q, none = sk.qk_norm_rope(c.q, None, c.qw, table=c.table, positions=c.positions[0])
    assert none is None and torch.equal(q, c.run()[0])
    outs = sk.qk_norm_rope_grad(c.dq, None, c.q, None, c.qw, table=c.table, positions=c.positions[0])
    full = c.grad()
    assert torch.equal(outs[0], full[0]) and outs[1] is None and outs[3] is None
    n = sum(c.q.shape[:2])
    assert torch.allclose(outs[2], full[2], rtol=1e-4, atol=1e-4 * n)


def test_empty():
    c = Case(0, 5, 2, 64)
    q, k = c.run()
    assert q.shape == (0, 5, 64) and k.shape == (0, 2, 64)
    outs = c.grad()
    assert not outs[2].any() and not outs[3].any()


def test_long_rows():
    """Token strides that carry the last tokens past 2^31 elements."""
    T, H, D, st = 40, 3, 64, (1 << 31) // 32 + 64
    buf = torch.empty(T * st, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(buf, (T, H, D), (st, D, 1))
    c = Case(T, H, 1, D)
    q.copy_(c.q)
    want = c.run()[0]
    got, _ = sk.qk_norm_rope(q, c.k, **c.kw_args(), q_out=q)
    assert torch.equal(got, want)


@pytest.mark.parametrize("pdl", [0, 1])
@pytest.mark.parametrize("T", [1, 64, 3000])
def test_same_bits_again_captured_and_on_a_stream(T, pdl):
    with sk.options(pdl=pdl):
        c = Case(T, 8, 2, 128)
        out = [torch.empty((T, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((T, 2, 128), dtype=torch.bfloat16, device="cuda")]
        din = [torch.empty_like(t) for t in out]
        dw = [torch.empty(128, device="cuda") for _ in range(2)]
        space = torch.empty(sk.qk_norm_rope_grad_workspace(T, 8, 2, 128), dtype=torch.uint8, device="cuda")

        def step(stream=None):
            c.run(q_out=out[0], k_out=out[1], stream=stream)
            c.grad(dq_in=din[0], dk_in=din[1], dq_weight=dw[0], dk_weight=dw[1], workspace=space, stream=stream)
            return out + din + dw
        first = [t.clone() for t in step()]
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, step()))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(first, out + din + dw))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in out + din + dw:
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out + din + dw))


def test_gradient_against_differences():
    """The loss <dq, y> in 64 bits along directions of x and of the weight."""
    c = Case(6, 3, 1, 32, R=20, dtype=torch.float32)
    cos, sin = c.angles()
    dx, _, dw, _ = c.grad()
    x, w, d = c.q.double().cpu(), c.qw.double().cpu(), c.dq.double().cpu()

    def loss(xx, ww):
        return (ref.heads(xx, ww, cos, sin, c.eps, False, torch.float64)[0] * d).sum().item()

    h = 1e-6
    g = torch.Generator().manual_seed(3)
    for _ in range(4):
        e = torch.randn(x.shape, generator=g, dtype=torch.double)
        diff = (loss(x + h * e, w) - loss(x - h * e, w)) / (2 * h)
        assert abs(diff - (dx.double().cpu() * e).sum().item()) <= 1e-3
        e = torch.randn(w.shape, generator=g, dtype=torch.double)
        diff = (loss(x, w + h * e) - loss(x, w - h * e)) / (2 * h)
        assert abs(diff - (dw.double().cpu() * e).sum().item()) <= 1e-3


def test_tensor_functions_refuse():
    c = Case(4, 3, 2, 32)
    with pytest.raises(ValueError):
        sk.qk_norm_rope(c.q, c.k, c.qw, c.kw, c.table, c.positions, eps=None)
    with pytest.raises(ValueError):
        sk.qk_norm_rope(c.q, c.k[:3], table=c.table, positions=c.positions)
    with pytest.raises(ValueError):
        sk.qk_norm_rope(c.q, c.k, table=c.table, positions=c.positions[:, :3])
    with pytest.raises(ValueError):
        sk.qk_norm_rope(c.q, c.k, table=c.table)
    with pytest.raises(TypeError):
        sk.qk_norm_rope(c.q.half(), None, table=c.table, positions=c.positions)
    with pytest.raises(TypeError):
        sk.qk_norm_rope(c.q, c.k, table=c.table, positions=c.positions.long())
    with pytest.raises(sk.SkinnyError):
        sk.qk_norm_rope(c.q, c.k, table=c.table[:, :3].contiguous(), positions=c.positions)       # an odd R
    with pytest.raises(sk.SkinnyError):
        c.run(q_out=c.k[:, :1].expand(4, 3, 32))
    with pytest.raises(sk.SkinnyError):
        c.grad(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
