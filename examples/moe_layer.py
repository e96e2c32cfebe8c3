"""The feed-forward part of a mixture-of-experts decoder layer at decode, from
the framework's calls alone:

    h       = x . W^T + s (x . A^T) . B^T      a shared projection, an adapter per request   lora_gemm
    ids, w  = top-k of softmax(h . R^T)        the router                                    skinny_router_bf16_topk
    hs      = h sorted by expert                                                             expert_dispatch
    g       = silu(hs . G_e^T) * (hs . U_e^T)  gate and up products, SwiGLU                  experts_gemm
    d       = g . D_e^T                        down product                                  experts_gemm
    y       = sum_j w_j d[pos_j]               back to the tokens                            expert_combine

and, for training the part around the experts, the gradients of the last step
and of the sort (expert_combine_grad, expert_combine without weights).

    python examples/moe_layer.py                  # checks one step against 64 bits, then times a captured step
    python examples/moe_layer.py --tokens 64 --hidden 7168 --experts 256 --inner 2048
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import latency_skinny_bf16_gb300 as sk  # noqa: E402


class Layer:
    """Weights, and the buffers one step writes."""

    def __init__(self, tokens, hidden, inner, experts, k, adapters, rank, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            b = shape[-1] ** -0.5
            return torch.empty(shape, device="cuda", dtype=torch.bfloat16).uniform_(-b, b, generator=g)

        self.k, self.experts = k, experts
        self.proj, self.router = weight(hidden, hidden), weight(experts, hidden)
        self.a, self.b = weight(adapters, rank, hidden), weight(adapters, hidden, rank)
        self.scales = torch.full((adapters,), 2.0, device="cuda")
        self.gate_up, self.down = weight(experts, 2 * inner, hidden), weight(experts, hidden, inner)
        rows = tokens * k

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.h, self.hs, self.act = empty(tokens, hidden), empty(rows, hidden), empty(rows, inner)
        self.logits, self.out = empty(tokens, experts, dtype=torch.float32), empty(tokens, hidden)
        self.d = empty(rows, hidden, dtype=torch.float32)
        self.weights, self.ids = empty(tokens, k, dtype=torch.float32), empty(tokens, k, dtype=torch.int32)
        self.pos, self.order = empty(tokens, k, dtype=torch.int32), empty(rows, dtype=torch.int32)
        self.offsets = empty(experts + 1, dtype=torch.int32)
        self.workspace = empty(sk.lora_workspace(tokens, hidden, rank, torch.bfloat16), dtype=torch.uint8)

    def step(self, x, adapter_ids):
        M, H = x.shape
        E = self.experts
        sk.lora_gemm(x, self.proj, self.a, self.b, adapter_ids, scales=self.scales, out=self.h, workspace=self.workspace)
        st = sk.skinny_router_bf16_topk(self.h.data_ptr(), H, self.router.data_ptr(), H, self.logits.data_ptr(), E, M, E,
                                        H, self.k, 1, self.weights.data_ptr(), self.k, self.ids.data_ptr(), self.k,
                                        torch.cuda.current_stream().cuda_stream)
        if st != sk.SKINNY_OK:
            raise sk.SkinnyError(st, "skinny_router_bf16_topk")
        sk.expert_dispatch(self.ids, E, x=self.h, xs=self.hs, pos=self.pos, order=self.order, offsets=self.offsets)
        sk.experts_gemm(self.hs, self.offsets, self.gate_up, out=self.act, activation="swiglu")
        sk.experts_gemm(self.act, self.offsets, self.down, out=self.d)
        return sk.expert_combine(self.d, self.pos, self.weights, out=self.out)

    def gradients(self, dy):
        """Of the combine and of the sort, as a training step around the experts takes them: (into the experts'
        rows, into the router's weights, into the tokens when the experts pass their rows' gradient through)."""
        dys, dweights = sk.expert_combine_grad(dy, self.d.to(dy.dtype), self.pos, self.weights)
        return dys, dweights, sk.expert_combine(dys, self.pos)


def reference(layer, x, adapter_ids):
    """The same step in 64 bits from the layer's own h, routing and activations: (h, act, out)."""
    f = torch.float64
    h = x.to(f) @ layer.proj.to(f).T
    for m, i in enumerate(adapter_ids.tolist()):
        if i >= 0:
            h[m] += 2.0 * (layer.b[i].to(f) @ (layer.a[i].to(f) @ x[m].to(f)))
    inner = layer.down.shape[2]
    act = torch.zeros((x.shape[0], layer.k, inner), dtype=f, device="cuda")
    out = torch.zeros_like(h)
    for m, ids in enumerate(layer.ids.tolist()):
        for j, e in enumerate(ids):
            gu = layer.gate_up[e].to(f) @ layer.h[m].to(f)
            act[m, j] = torch.nn.functional.silu(gu[:inner]) * gu[inner:]
            out[m] += float(layer.weights[m, j]) * (layer.down[e].to(f) @ layer.act[layer.pos[m, j]].to(f))
    return h, act, out


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--hidden", type=int, default=2880)
    p.add_argument("--inner", type=int, default=1440)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--topk", type=int, default=4)
    p.add_argument("--adapters", type=int, default=6)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--replays", type=int, default=50)
    a = p.parse_args(argv)
    if sk.skinny_init(torch.cuda.current_device()) != sk.SKINNY_OK:
        raise SystemExit("no GB300")
    layer = Layer(a.tokens, a.hidden, a.inner, a.experts, a.topk, a.adapters, a.rank)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    adapter_ids = torch.randint(-1, a.adapters, (a.tokens,), generator=g, device="cuda").to(torch.int32)

    y = layer.step(x, adapter_ids)
    h, act, out = reference(layer, x, adapter_ids)
    half = 2.0 ** -8                                   # half a step of bf16
    got_act = layer.act[layer.pos.long()].double()
    for name, got, want in (("h", layer.h.double(), h), ("act", got_act, act), ("y", y.double(), out)):
        off = float(((got - want).abs() - half * want.abs()).max() / want.abs().max())
        print(f"{name:4s} largest error past half a step of bf16, of its largest value: {max(off, 0.0):.1e}")
        if off > 1e-3:
            raise SystemExit(f"{name} is off")
    dy = torch.randn(a.tokens, a.hidden, generator=g, device="cuda")
    dys, dweights, dx = layer.gradients(dy)
    want = dy.double() * layer.weights.double().sum(1, keepdim=True)
    print(f"dx   largest error: {float((dx.double() - want).abs().max()):.1e}")
    slope = float((dweights.double() * layer.weights).sum() - (dy.double() * out).sum())
    print(f"<dweights, weights> - <dy, y>: {slope:.1e}")

    with sk.options(pdl=1):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer.step(x, adapter_ids)
    y0 = y.clone()
    for t in (layer.h, layer.logits, layer.weights, layer.hs, layer.act, layer.d, layer.out):
        t.fill_(float("nan"))                          # nothing of the eager step is left to the captured one
    for t in (layer.ids, layer.pos, layer.order, layer.offsets):
        t.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    if not torch.equal(layer.out, y0):
        raise SystemExit("the captured step differs from the eager one")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.replays):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    touched = layer.ids.unique().numel()
    print(f"one captured step: {1e3 * start.elapsed_time(end) / a.replays:.1f} us, {a.tokens} tokens, {touched} of "
          f"{a.experts} experts")


if __name__ == "__main__":
    main()
