"""The projections of a dense decoder layer and what stands between them and
attention, from the framework's calls alone:

    qkv  = x . Wqkv^T + b                         linear
    q, k = turned(norm(q)), turned(norm(k))       qk_norm_rope, views into qkv's rows
    h    = x + o . Wo^T                           linear with a residual (attention's place: o is q here)
    g    = silu(h . G^T) * (h . U^T)              linear, both projections of the gated block
    y    = h + g . D^T                            linear with a residual

and the backward pass of the gated block and of its down product (linear_grad).

    python examples/dense_layer.py                    # checks one step against 64 bits, then times a captured step
    python examples/dense_layer.py --tokens 64 --hidden 7168 --inner 2048 --heads 64 --kv 8
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import latency_skinny_bf16_gb300 as sk  # noqa: E402

POSITIONS = 4096


class Layer:
    """Weights, and the buffers one step writes."""

    def __init__(self, tokens, hidden, inner, heads, kv, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            b = shape[-1] ** -0.5
            return torch.empty(shape, device="cuda", dtype=torch.bfloat16).uniform_(-b, b, generator=g)

        def empty(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

        self.heads, self.kv, self.dim, self.inner = heads, kv, dim, inner
        rows = (heads + 2 * kv) * dim
        self.wqkv, self.bqkv, self.wo = weight(rows, hidden), weight(rows), weight(hidden, heads * dim)
        self.gate_up, self.down = weight(2 * inner, hidden), weight(hidden, inner)
        self.qw, self.kw = 1 + weight(dim), 1 + weight(dim)
        angle = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * \
            1e6 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.table = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        self.qkv, self.q, self.k = empty(tokens, heads + 2 * kv, dim), empty(tokens, heads, dim), empty(tokens, kv, dim)
        self.h, self.act, self.pre, self.y = empty(tokens, hidden), empty(tokens, inner), empty(tokens, 2 * inner), empty(tokens, hidden)

    def step(self, x, positions):
        T = x.shape[0]
        sk.linear(x, self.wqkv, bias=self.bqkv, out=self.qkv.view(T, -1))
        q, k = self.qkv[:, :self.heads], self.qkv[:, self.heads:self.heads + self.kv]
        sk.qk_norm_rope(q, k, self.qw, self.kw, self.table, positions, q_out=self.q, k_out=self.k)
        sk.linear(self.q.view(T, -1), self.wo, residual=x, out=self.h)
        sk.linear(self.h, self.gate_up, activation="swiglu", out=self.act, pre=self.pre)
        return sk.linear(self.act, self.down, residual=self.h, out=self.y)

    def gradients(self, dy):
        """Of the gated block and its down product: (into h, into gate_up, into down)."""
        dact, ddown, _ = sk.linear_grad(dy, self.act, self.down)
        dh, dgate_up, _ = sk.linear_grad(dact, self.h, self.gate_up, pre=self.pre, activation="swiglu")
        return dh + dy, dgate_up, ddown


def reference(layer, x, positions):
    """The same step in 64 bits, each part from the layer's own input to it: (qkv, q, h, act, y)."""
    f = torch.float64
    T = x.shape[0]
    qkv = x.to(f) @ layer.wqkv.to(f).T + layer.bqkv.to(f)
    q = layer.qkv[:, :layer.heads].to(f)
    n = q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt() * layer.qw.to(f)
    half = layer.dim // 2
    c, s = layer.table[positions.long()][:, None].to(f).split(half, dim=2)
    turned = torch.cat([n[..., :half] * c - n[..., half:] * s, n[..., half:] * c + n[..., :half] * s], dim=2)
    h = x.to(f) + layer.q.view(T, -1).to(f) @ layer.wo.to(f).T
    gu = layer.h.to(f) @ layer.gate_up.to(f).T
    act = torch.nn.functional.silu(gu[:, :layer.inner]) * gu[:, layer.inner:]
    return qkv, turned, h, act, layer.h.to(f) + layer.act.to(f) @ layer.down.to(f).T


def gradients(layer, dy):
    """`Layer.gradients` in 64 bits."""
    f = torch.float64
    h, gate_up, down = (t.to(f).requires_grad_(True) for t in (layer.h, layer.gate_up, layer.down))
    gu = h @ gate_up.T
    y = h + (torch.nn.functional.silu(gu[:, :layer.inner]) * gu[:, layer.inner:]) @ down.T
    return torch.autograd.grad(y, [h, gate_up, down], dy.to(f))


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--hidden", type=int, default=2880)
    p.add_argument("--inner", type=int, default=1440)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv", type=int, default=8)
    p.add_argument("--dim", type=int, default=64)
    p.add_argument("--replays", type=int, default=50)
    a = p.parse_args(argv)
    if sk.skinny_init(torch.cuda.current_device()) != sk.SKINNY_OK:
        raise SystemExit("no GB300")
    layer = Layer(a.tokens, a.hidden, a.inner, a.heads, a.kv, a.dim)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    positions = torch.randint(0, POSITIONS, (a.tokens,), generator=g, device="cuda", dtype=torch.int32)

    layer.step(x, positions)
    half = 2.0 ** -8                                   # half a step of bf16

    def report(name, got, want, limit):
        off = float(((got.double() - want).abs() - half * want.abs()).max() / want.abs().max())
        print(f"{name:9s} largest error past half a step of bf16, of its largest value: {max(off, 0.0):.1e}")
        if not off <= limit:
            raise SystemExit(f"{name} is off")

    got = (layer.qkv.view(a.tokens, -1), layer.q, layer.h, layer.act, layer.y)
    for name, t, want in zip(("qkv", "q", "h", "act", "y"), got, reference(layer, x, positions)):
        report(name, t, want, 1e-3)
    dy = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    for name, t, want in zip(("dh", "dgate_up", "ddown"), layer.gradients(dy), gradients(layer, dy)):
        report(name, t, want, 2e-2)                    # through what the steps between round to bf16

    with sk.options(pdl=1):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer.step(x, positions)
    y0 = layer.y.clone()
    for t in (layer.qkv, layer.q, layer.k, layer.h, layer.act, layer.pre, layer.y):
        t.fill_(float("nan"))                          # nothing of the eager step is left to the captured one
    graph.replay()
    torch.cuda.synchronize()
    if not torch.equal(layer.y, y0):
        raise SystemExit("the captured step differs from the eager one")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.replays):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"one captured step: {1e3 * start.elapsed_time(end) / a.replays:.1f} us, {a.tokens} tokens")


if __name__ == "__main__":
    main()
