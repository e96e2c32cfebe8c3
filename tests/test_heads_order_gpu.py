"""Positions, axes, table and weights that a call just before writes: heads see them in the stream's order, whatever
starts early."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk

pytestmark = pytest.mark.gpu

WRITERS = ("positions", "axes", "table", "weights")


@pytest.mark.parametrize("last", WRITERS)
@pytest.mark.parametrize("T,Hq,Hk,D,dtype", [(1, 4, 1, 128, torch.bfloat16), (40, 8, 2, 64, torch.bfloat16), (300, 3, 3, 61, torch.bfloat16),
                                             (300, 8, 8, 72, torch.float32)])
@pytest.mark.parametrize("pdl", [1, 2])
def test_inputs_that_a_call_just_before_writes(T, Hq, Hk, D, dtype, last, pdl):
    g = torch.Generator(device="cuda").manual_seed(T)
    R, axes, rounds = 16, 8, 6
    P = axes * T

    def new(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    def ids(n):
        return torch.randint(0, 5, (n, 1), generator=g, device="cuda", dtype=torch.int32)

    def buf(*shape, dtype=dtype):
        return torch.empty(shape, device="cuda", dtype=dtype)

    sources = [dict(positions=ids(P), axes=ids(R // 2), table=new(P, 64), weights=new(2, 64)) for _ in range(rounds)]
    angles, scales = new(R, 64) * 0.1, new(D, 64) * 0.1
    q, k, dq, dk = (torch.randn((T, h, D), generator=g, device="cuda").to(dtype) for h in (Hq, Hk, Hq, Hk))
    positions, pair_axis = buf(axes, T, dtype=torch.int32), buf(R // 2, dtype=torch.int32)
    table, weights = buf(P, R, dtype=torch.float32), buf(2, D)
    spare = [buf(n, dtype=torch.int32) for n in (P, 6, R // 2, 6)]
    outs = [[buf(T, Hq, D), buf(T, Hk, D), buf(T, Hq, D), buf(T, Hk, D), buf(D, dtype=torch.float32), buf(D, dtype=torch.float32)]
            for _ in range(rounds)]
    space = buf(sk.qk_norm_rope_grad_workspace(T, Hq, Hk, D), dtype=torch.uint8)
    write = {
        "positions": lambda s: sk.expert_dispatch(s, 5, pos=spare[0].view(P, 1), order=positions.view(P), offsets=spare[1]),
        "axes": lambda s: sk.expert_dispatch(s, 5, pos=spare[2].view(-1, 1), order=pair_axis, offsets=spare[3]),
        "table": lambda s: sk.linear(s, angles, out=table),
        "weights": lambda s: sk.linear(s, scales, out=weights),
    }

    def run(wait):
        for t in (positions, pair_axis, table, weights):
            t.zero_()
        wait()
        args = dict(q_weight=weights[0], k_weight=weights[1], table=table, positions=positions, pair_axis=pair_axis)
        for source, out in zip(sources, outs):
            for name in sorted(WRITERS, key=lambda n: n == last):
                write[name](source[name])
                wait()
            sk.qk_norm_rope(q, k, **args, q_out=out[0], k_out=out[1])
            wait()
            write[last](source[last])
            wait()
            sk.qk_norm_rope_grad(dq, dk, q, k, **args, dq_in=out[2], dk_in=out[3], dq_weight=out[4], dk_weight=out[5],
                                 workspace=space)
            wait()
        torch.cuda.synchronize()
        return [t.clone() for out in outs for t in out]

    with sk.options(pdl=pdl):
        want = run(torch.cuda.synchronize)
        assert any(not torch.equal(a, b) for a, b in zip(want[:6], want[6:12]))
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
    assert sk.skinny_get_device_status() == 0


@pytest.mark.parametrize("T", [300, 3000, 9000])
@pytest.mark.parametrize("pdl", [1, 2])
def test_positions_renewed_while_their_readers_run(T, pdl):
    """The calls follow each other without a wait: the one that renews positions lets its successor start before it
    has waited for its predecessor, so heads of two calls share SMs."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rounds, Hq, Hk, D = 24, 8, 2, 64
    ids = [torch.randint(0, 7, (T, 1), generator=g, device="cuda", dtype=torch.int32) for _ in range(rounds)]
    q, k = (torch.randn((T, h, D), generator=g, device="cuda").bfloat16() for h in (Hq, Hk))
    angle = torch.arange(T, device="cuda")[:, None] * 0.37 ** torch.arange(D // 2, device="cuda")
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    positions, spare, counts = (torch.zeros(n, device="cuda", dtype=torch.int32) for n in (T, T, 8))
    outs = [torch.empty((T, Hq, D), device="cuda", dtype=torch.bfloat16) for _ in range(rounds)]
    ko = torch.empty((T, Hk, D), device="cuda", dtype=torch.bfloat16)

    def run(wait):
        for i, out in zip(ids, outs):
            sk.expert_dispatch(i, 7, pos=spare.view(T, 1), order=positions, offsets=counts)
            wait()
            sk.qk_norm_rope(q, k, table=table, positions=positions, q_out=out, k_out=ko)
            wait()
        torch.cuda.synchronize()
        return [t.clone() for t in outs]

    with sk.options(pdl=pdl):
        want = run(torch.cuda.synchronize)
        for _ in range(10):
            assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i, out in zip(ids, outs):
                sk.expert_dispatch(i, 7, pos=spare.view(T, 1), order=positions, offsets=counts)
                sk.qk_norm_rope(q, k, table=table, positions=positions, q_out=out, k_out=ko)
        for _ in range(10):
            for t in outs:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
