"""Heads of queries, keys and values by turns, [T, H, 3, D]: in place and into a buffer of the same order, against 64
bits with the bounds of the other layouts."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk
import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,R", [(1, 4, 64, 64), (40, 8, 128, 128), (300, 3, 61, 60), (2000, 5, 72, 36), (3, 2, 333, 332)])
@pytest.mark.parametrize("first", ["tokens", "heads"])
def test_by_turns(first, T, H, D, R, interleaved, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    shape = (T, H, 3, D) if first == "tokens" else (H, T, 3, D)

    def rows():
        buf = torch.randn(shape, generator=g, device="cuda").to(dtype)
        q, k, v = (buf[:, :, i] if first == "tokens" else buf[:, :, i].transpose(0, 1) for i in range(3))
        return q, k, v

    (q, k, v), (dq, dk, dv) = rows(), rows()
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    angle = torch.arange(500, device="cuda")[:, None] * 0.8 ** torch.arange(R // 2, device="cuda")
    args = dict(q_weight=w[0], k_weight=w[1], table=torch.cat([angle.cos(), angle.sin()], 1).float(), interleaved=interleaved,
                positions=torch.randint(0, 500, (T,), generator=g, device="cuda", dtype=torch.int32))
    rest, out = v.clone(), rows()
    kept = out[2].clone()
    cos, sin = ref.angles(args["table"], args["positions"], None, T)
    sk.qk_norm_rope(q, k, **args, q_out=out[0], k_out=out[1])
    again = [t.clone() for t in sk.qk_norm_rope_grad(dq, dk, q, k, **args)]
    for i, (x, d) in enumerate(((q, dq), (k, dk))):
        ref.check(out[i], *ref.heads(x, w[i], cos, sin, 1e-6, interleaved, dtype))
        dx, dw = ref.heads_grad(d, x, w[i], cos, sin, 1e-6, interleaved, dtype)
        ref.check(again[i], *dx)
        ref.check(again[2 + i], *dw)
    assert torch.equal(out[2], kept)
    got = sk.qk_norm_rope_grad(dq, dk, q, k, **args, dq_in=dq, dk_in=dk)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    first_out = [t.clone() for t in out[:2]]
    got = sk.qk_norm_rope(q, k, **args, q_out=q, k_out=k)
    assert all(torch.equal(a, b) for a, b in zip(got, first_out)) and torch.equal(v, rest)
