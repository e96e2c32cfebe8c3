"""Dispatch, the experts' products and combine one behind the other, as a layer
runs them: each may start while the one before it still runs, so its buffers
are filled and the tokens change before every replay."""
import pytest
import torch

import experts_ref as ref
import latency_skinny_bf16_gb300 as sk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _init():
    assert sk.skinny_init(0) == sk.SKINNY_OK
    yield
    assert sk.skinny_get_device_status() == 0


@pytest.mark.parametrize("pdl", [1, 2])
@pytest.mark.parametrize("T,k,E,H,inner", [(16, 4, 32, 512, 264), (64, 8, 16, 1024, 1536), (900, 4, 24, 264, 136), (13, 3, 9, 257, 131),
                                           (1, 4, 8, 2880, 2880)])
def test_layer(T, k, E, H, inner, pdl):
    g = torch.Generator(device="cuda").manual_seed(T)

    def weight(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

    gate_up, down = weight(E, 2 * inner, H), weight(E, H, inner)
    steps = []
    for s in range(3):
        ids, w = ref.routing(T, k, E, seed=s, drop=0.2 * (s % 2))
        steps.append((torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), weight(T, H), weight(T, H)))
    ids, wt, x, dy = (t.clone() for t in steps[0])
    n = T * k

    def buffer(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    xs, act, d, y = buffer(n, H), buffer(n, inner), buffer(n, H), buffer(T, H)
    dys, dx, dw = buffer(n, H), buffer(T, H), buffer(T, k, dtype=torch.float32)
    pos, order, off = buffer(T, k, dtype=torch.int32), buffer(n, dtype=torch.int32), buffer(E + 1, dtype=torch.int32)
    buffers = (xs, act, d, y, dys, dx, dw, pos, order, off)

    def layer():
        sk.expert_dispatch(ids, E, x=x, xs=xs, pos=pos, order=order, offsets=off)
        sk.experts_gemm(xs, off, gate_up, out=act, activation="swiglu")
        sk.experts_gemm(act, off, down, out=d)
        sk.expert_combine(d, pos, wt, out=y)
        sk.expert_combine_grad(dy, d, pos, wt, dys=dys, dweights=dw)
        sk.expert_combine(dys, pos, out=dx)

    def load(step):
        for to, v in zip((ids, wt, x, dy), step):
            to.copy_(v)
        for b in buffers:
            b.view(torch.uint8).fill_(0xFF)    # NaN, and positions and offsets that are refused

    want = []
    for step in steps:
        load(step)
        layer()
        torch.cuda.synchronize()
        want.append([b.clone() for b in buffers])
        assert torch.isfinite(y).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()
    with sk.options(pdl=pdl):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer()
        for run in (layer, graph.replay):
            for i in (1, 2, 0, 1):
                load(steps[i])
                run()
                torch.cuda.synchronize()
                for got, v in zip(buffers, want[i]):
                    assert torch.equal(got.view(torch.uint8), v.view(torch.uint8))
        del graph
