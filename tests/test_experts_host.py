"""Host-side tests of include/skinny_experts.h: every argument error is
reported before any CUDA call.  No GPU needed, no kernel launched."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk

A, B, C, D, F, G = (0x7F0000000000 + i * 0x10000000 for i in range(6))   # fake, aligned; never dereferenced
INVALID, UNSUPPORTED, MISALIGNED = sk.SKINNY_ERR_INVALID_VALUE, sk.SKINNY_ERR_UNSUPPORTED, sk.SKINNY_ERR_MISALIGNED


def dispatch(ids=A, ldid=4, X=B, ldx=64, T=8, k=4, E=16, H=64, dtype=0, pos=C, order=C + 4096, offsets=D, Xs=F, ldxs=64):
    return sk.skinny_expert_dispatch(ids, ldid, X, ldx, T, k, E, H, dtype, pos, order, offsets, Xs, ldxs)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(k=-1), INVALID), (dict(E=0), INVALID), (dict(H=-1), INVALID),
    (dict(k=65, ldid=65), UNSUPPORTED), (dict(E=8193), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(H=(1 << 20) + 1, ldx=1 << 21, ldxs=1 << 21), UNSUPPORTED),
    (dict(ids=0), INVALID), (dict(pos=0), INVALID), (dict(offsets=0), INVALID), (dict(Xs=0), INVALID),
    (dict(ldid=3), INVALID), (dict(ldx=63), INVALID), (dict(ldxs=63), INVALID), (dict(dtype=2), INVALID),
    (dict(ids=A + 2), MISALIGNED), (dict(pos=C + 1), MISALIGNED), (dict(order=C + 4098), MISALIGNED),
    (dict(offsets=D + 2), MISALIGNED), (dict(X=B + 1), MISALIGNED), (dict(Xs=F + 1), MISALIGNED),
    (dict(dtype=1, X=B + 2), MISALIGNED),
    (dict(Xs=B + 64), INVALID), (dict(pos=A), INVALID), (dict(order=C), INVALID), (dict(offsets=C), INVALID),
    (dict(offsets=B), INVALID), (dict(pos=F + 128), INVALID),
])
def test_dispatch_refusals(kw, expect):
    assert dispatch(**kw) == expect


def combine(Ys=A, ldys=64, rows=32, pos=B, weights=C, ldw=4, T=8, k=4, H=64, it=0, ot=0, Y=D, ldy=64):
    return sk.skinny_expert_combine(Ys, ldys, rows, pos, weights, ldw, T, k, H, it, ot, Y, ldy)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=0), sk.SKINNY_OK), (dict(H=0), sk.SKINNY_OK),
    (dict(T=-1), INVALID), (dict(k=-1), INVALID), (dict(H=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(it=2), INVALID), (dict(ot=-1), INVALID), (dict(k=65, ldw=65), UNSUPPORTED),
    (dict(Ys=0), INVALID), (dict(pos=0), INVALID), (dict(Y=0), INVALID), (dict(ldys=63), INVALID),
    (dict(ldy=63), INVALID), (dict(ldw=3), INVALID), (dict(Y=D + 1), MISALIGNED), (dict(Ys=A + 1), MISALIGNED),
    (dict(pos=B + 2), MISALIGNED), (dict(weights=C + 2), MISALIGNED), (dict(ot=1, Y=D + 2), MISALIGNED),
    (dict(Y=A + 128), INVALID), (dict(Y=B), INVALID), (dict(Y=C), INVALID),
])
def test_combine_refusals(kw, expect):
    assert combine(**kw) == expect


def grad(dY=A, lddy=64, Ys=B, ldys=64, rows=32, pos=C, weights=C + 4096, ldw=4, T=8, k=4, H=64, dt=0, dYs=D, lddys=64,
         dw=F, lddw=4):
    return sk.skinny_expert_combine_grad(dY, lddy, Ys, ldys, rows, pos, weights, ldw, T, k, H, dt, dYs, lddys, dw, lddw)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=0), sk.SKINNY_OK), (dict(k=0), sk.SKINNY_OK), (dict(T=-1), INVALID), (dict(H=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(dt=3), INVALID), (dict(k=65, ldw=65, lddw=65), UNSUPPORTED),
    (dict(dY=0), INVALID), (dict(Ys=0), INVALID), (dict(pos=0), INVALID), (dict(dYs=0), INVALID),
    (dict(lddy=63), INVALID), (dict(ldys=63), INVALID), (dict(lddys=63), INVALID), (dict(ldw=3), INVALID),
    (dict(lddw=3), INVALID), (dict(dY=A + 1), MISALIGNED), (dict(Ys=B + 1), MISALIGNED), (dict(dYs=D + 1), MISALIGNED),
    (dict(pos=C + 2), MISALIGNED), (dict(dw=F + 2), MISALIGNED), (dict(weights=C + 4098), MISALIGNED),
    (dict(dYs=A), INVALID), (dict(dYs=B), INVALID), (dict(dw=D), INVALID), (dict(dw=C), INVALID),
    (dict(dw=C + 4096), INVALID),
])
def test_combine_grad_refusals(kw, expect):
    assert grad(**kw) == expect


def test_tensor_functions_refuse_what_they_cannot_take():
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        sk.expert_dispatch(ids, 8)                       # not on a GPU
    with pytest.raises(ValueError):
        sk.expert_combine(torch.zeros((8, 4)), ids)


def experts(Xs=A, ldx=64, rows=32, offsets=B, W=C, ldw=64, ldwe=64 * 48, E=8, N=48, K=64, act=0, ot=0, Y=D, ldy=48):
    return sk.skinny_experts_gemm_bf16(Xs, ldx, rows, offsets, W, ldw, ldwe, E, N, K, act, ot, Y, ldy)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), sk.SKINNY_OK), (dict(N=0), sk.SKINNY_OK),
    (dict(E=0), INVALID), (dict(rows=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(act=2), INVALID),
    (dict(ot=2), INVALID), (dict(E=1025), UNSUPPORTED), (dict(N=(1 << 20) + 1, ldy=1 << 21), UNSUPPORTED),
    (dict(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), UNSUPPORTED),
    (dict(Xs=0), INVALID), (dict(offsets=0), INVALID), (dict(W=0), INVALID), (dict(Y=0), INVALID),
    (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(ldwe=64 * 48 - 1), INVALID), (dict(ldy=47), INVALID),
    (dict(act=1), INVALID),                              # the stride of an expert holds 48 rows, not 96
    (dict(Xs=A + 1), MISALIGNED), (dict(W=C + 1), MISALIGNED), (dict(offsets=B + 2), MISALIGNED),
    (dict(Y=D + 1), MISALIGNED), (dict(ot=1, Y=D + 2), MISALIGNED),
    (dict(Y=A), INVALID), (dict(Y=C + 7 * 64 * 48 * 2), INVALID), (dict(Y=B), INVALID),
])
def test_experts_gemm_refusals(kw, expect):
    assert experts(**kw) == expect


def lora(X=A, ldx=64, W=B, ldw=64, Aw=C, lda=64, ldae=8 * 64, Bw=D, ldb=8, ldbe=48 * 8, ids=F, ranks=F + 4096,
         scales=F + 8192, L=4, R=8, Y=G, ldy=48, M=5, N=48, K=64, ot=0, ws=G + (1 << 20), wsb=1 << 20):
    return sk.skinny_lora_gemm_bf16(X, ldx, W, ldw, Aw, lda, ldae, Bw, ldb, ldbe, ids, ranks, scales, L, R, Y, ldy, M, N,
                                    K, ot, ws, wsb)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=0), sk.SKINNY_OK), (dict(N=0), sk.SKINNY_OK),
    (dict(L=-1), INVALID), (dict(R=-1), INVALID), (dict(ot=2), INVALID), (dict(M=-1), INVALID),
    (dict(R=257, ldb=257), UNSUPPORTED), (dict(M=65), UNSUPPORTED),
    (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(Aw=0), INVALID), (dict(Bw=0), INVALID), (dict(ids=0), INVALID),
    (dict(Y=0), INVALID), (dict(ws=0), INVALID), (dict(ot=1, wsb=5 * 32 * 6 - 1), INVALID), (dict(ot=0, wsb=5 * 32 * 6), INVALID),
    (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(lda=63), INVALID), (dict(ldb=7), INVALID),
    (dict(ldae=511), INVALID), (dict(ldbe=383), INVALID), (dict(ldy=47), INVALID),
    (dict(X=A + 1), MISALIGNED), (dict(Aw=C + 1), MISALIGNED), (dict(Bw=D + 1), MISALIGNED), (dict(ids=F + 2), MISALIGNED),
    (dict(ranks=F + 4098), MISALIGNED), (dict(scales=F + 8193), MISALIGNED), (dict(ws=G + (1 << 20) + 8), MISALIGNED),
    (dict(Y=G + 1), MISALIGNED), (dict(ot=1, Y=G + 2), MISALIGNED),
    (dict(Y=A), INVALID), (dict(Y=B), INVALID), (dict(Y=C), INVALID), (dict(Y=D), INVALID), (dict(Y=F), INVALID),
    (dict(Y=F + 4096), INVALID), (dict(Y=F + 8192), INVALID), (dict(ws=A), INVALID), (dict(ws=D), INVALID),
    (dict(ws=G), INVALID), (dict(ws=F), INVALID),
])
def test_lora_refusals(kw, expect):
    assert lora(**kw) == expect


def test_lora_workspace():
    # six bytes for each of the columns of V, in whole steps of 32; bf16: the fp32 projection too
    assert sk.skinny_lora_workspace(5, 48, 8, sk.SKINNY_F32) == 5 * 32 * 6
    assert sk.skinny_lora_workspace(5, 48, 33, sk.SKINNY_BF16) == 5 * 64 * 6 + 5 * 48 * 4
    for bad in ((65, 48, 8, 0), (5, -1, 8, 0), (5, 48, 257, 0), (5, 48, 8, 2), (-1, 48, 8, 0)):
        assert sk.skinny_lora_workspace(*bad) == 0
