"""Run one operator around the router a few times, for a profiler.

    python -m latency_skinny_bf16_gb300.profile_op --op experts --T 16 --k 8 --E 64 --N 2048 --K 7168 --act swiglu

``--op`` is dispatch, combine, combine_grad, experts or lora; ``--calls`` calls
run, alternating between two sets of inputs (together larger than L2 at sizes
worth profiling).  Prints the algorithmic bytes of a call: each input read
once, each output written once, the weights of the experts or adapters that
occur.
"""
from __future__ import annotations

import argparse
import json

import torch

import latency_skinny_bf16_gb300 as sk


def routing(a, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randn(a.T, a.E, generator=g, device="cuda").topk(a.k, dim=1).indices.int()
    return ids, sk.expert_dispatch(ids, a.E)


def rand(*shape, dtype=torch.bfloat16, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").uniform_(-scale, scale)


def prepare(a, seed):
    """(the call, its algorithmic bytes)."""
    if a.op == "lora":
        x, w = rand(a.T, a.K), rand(a.N, a.K, scale=a.K ** -0.5)
        la, lb = rand(a.E, a.R, a.K, scale=a.K ** -0.5), rand(a.E, a.N, a.R, scale=a.R ** -0.5)
        ids = torch.arange(a.T, device="cuda", dtype=torch.int32) % a.E
        used = min(a.T, a.E)
        return (lambda: sk.lora_gemm(x, w, la, lb, ids),
                2 * (a.N * a.K + used * a.R * (a.N + a.K) + a.T * a.K) + 4 * a.T * a.N)
    ids, (_, pos, _, offsets) = routing(a, seed)
    rows = a.T * a.k
    if a.op == "experts":
        wrows = 2 * a.N if a.act == "swiglu" else a.N
        xs, w = rand(rows, a.K), rand(a.E, wrows, a.K, scale=a.K ** -0.5)
        out = torch.empty((rows, a.N), dtype=torch.bfloat16, device="cuda")
        touched = int((offsets[1:] > offsets[:-1]).sum())
        return (lambda: sk.experts_gemm(xs, offsets, w, out=out, activation=a.act),
                2 * (touched * wrows * a.K + rows * (a.K + a.N)))
    x, ys, weights = rand(a.T, a.N), rand(rows, a.N), torch.rand((a.T, a.k), device="cuda")
    if a.op == "dispatch":
        return lambda: sk.expert_dispatch(ids, a.E, x=x, xs=ys), 2 * a.N * (a.T + rows) + 12 * rows
    if a.op == "combine":
        return lambda: sk.expert_combine(ys, pos, weights, out=x), 2 * a.N * (a.T + rows) + 8 * rows
    dys = torch.empty_like(ys)
    return (lambda: sk.expert_combine_grad(x, ys, pos, weights, dys=dys),
            2 * a.N * (a.T + 2 * rows) + 12 * rows)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--op", choices=["dispatch", "combine", "combine_grad", "experts", "lora"], required=True)
    p.add_argument("--T", type=int, default=16, help="tokens")
    p.add_argument("--k", type=int, default=8, help="experts per token")
    p.add_argument("--E", type=int, default=64, help="experts, or adapters")
    p.add_argument("--N", type=int, default=2048, help="outputs; the rows' width for dispatch and combine")
    p.add_argument("--K", type=int, default=7168)
    p.add_argument("--R", type=int, default=16, help="rank of the adapters")
    p.add_argument("--act", choices=["none", "swiglu"], default="none")
    p.add_argument("--calls", type=int, default=6)
    a = p.parse_args(argv)
    assert sk.skinny_init(0) == sk.SKINNY_OK
    calls = [prepare(a, seed) for seed in (1, 2)]
    for i in range(a.calls):
        calls[i % 2][0]()
    torch.cuda.synchronize()
    code = sk.skinny_get_device_status()
    if code:
        raise RuntimeError(f"device status {code:#x}")
    print(json.dumps({**vars(a), "algorithmic_bytes": [c[1] for c in calls]}))


if __name__ == "__main__":
    main()
