"""Host-side tests of include/skinny_layer.h: every argument error is reported
before any CUDA call.  No GPU needed, no kernel launched."""
import ctypes

import pytest
import torch

import latency_skinny_bf16_gb300 as sk

A, B, C, D, F, G, H = (0x7F0000000000 + i * 0x10000000 for i in range(7))   # fake, aligned; never dereferenced
INVALID, UNSUPPORTED, MISALIGNED = sk.SKINNY_ERR_INVALID_VALUE, sk.SKINNY_ERR_UNSUPPORTED, sk.SKINNY_ERR_MISALIGNED
MAX = 1 << 20


def linear(X=A, ldx=64, W=B, ldw=64, bias=C, R=D, ldr=48, Y=F, ldy=48, Z=G, ldz=96, M=5, N=48, K=64, act=0, ot=0, ws=H,
           wsb=1 << 24):
    return sk.skinny_linear_bf16(X, ldx, W, ldw, bias, R, ldr, Y, ldy, Z, ldz, M, N, K, act, ot, ws, wsb)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=0), sk.SKINNY_OK), (dict(N=0), sk.SKINNY_OK),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(ot=2), INVALID), (dict(N=MAX + 1), UNSUPPORTED), (dict(K=MAX + 1), UNSUPPORTED),
    (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(Y=0), INVALID),
    (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(ldr=47), INVALID), (dict(ldy=47), INVALID), (dict(ldz=47), INVALID),
    (dict(act=1, ldz=95), INVALID), (dict(act=4, ldz=95), INVALID),
    (dict(X=A + 1), MISALIGNED), (dict(W=B + 1), MISALIGNED), (dict(bias=C + 1), MISALIGNED), (dict(R=D + 1), MISALIGNED),
    (dict(Y=F + 1), MISALIGNED), (dict(Z=G + 1), MISALIGNED), (dict(ot=1, Y=F + 2), MISALIGNED), (dict(ot=1, R=D + 2), MISALIGNED),
    (dict(Y=A), INVALID), (dict(Y=B + 64), INVALID), (dict(Y=C), INVALID), (dict(Y=D + 2), INVALID), (dict(Y=G), INVALID),
    (dict(Y=D, ldy=49), INVALID), (dict(Z=A), INVALID), (dict(Z=B), INVALID), (dict(Z=C), INVALID), (dict(Z=D), INVALID),
])
def test_linear_refusals(kw, expect):
    assert linear(**kw) == expect


def grad(dY=A, lddy=48, X=B, ldx=64, W=C, ldw=64, Z=D, ldz=96, dX=F, lddx=64, dW=G, lddw=64, db=G + (1 << 20), M=5, N=48, K=64,
         act=1, ws=H, wsb=1 << 24):
    return sk.skinny_linear_grad_bf16(dY, lddy, X, ldx, W, ldw, Z, ldz, dX, lddx, dW, lddw, db, M, N, K, act, ws, wsb)


@pytest.mark.parametrize("kw,expect", [
    (dict(dX=0, dW=0, db=0), sk.SKINNY_OK), (dict(M=0, dW=0, db=0), sk.SKINNY_OK), (dict(N=0, dX=0), sk.SKINNY_OK),
    (dict(K=0, db=0), sk.SKINNY_OK),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(act=5), INVALID),
    (dict(N=MAX + 1), UNSUPPORTED), (dict(K=MAX + 1), UNSUPPORTED),
    (dict(dY=0), INVALID), (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(Z=0), INVALID), (dict(ws=0), INVALID), (dict(wsb=64), INVALID),
    (dict(lddy=47), INVALID), (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(ldz=95), INVALID), (dict(lddx=63), INVALID),
    (dict(lddw=63), INVALID),
    (dict(dY=A + 1), MISALIGNED), (dict(X=B + 1), MISALIGNED), (dict(W=C + 1), MISALIGNED), (dict(Z=D + 1), MISALIGNED),
    (dict(dX=F + 1), MISALIGNED), (dict(dW=G + 1), MISALIGNED), (dict(db=G + (1 << 20) + 2), MISALIGNED), (dict(ws=H + 8), MISALIGNED),
    (dict(dX=A), INVALID), (dict(dX=B), INVALID), (dict(dX=C), INVALID), (dict(dX=D), INVALID), (dict(dX=G), INVALID), (dict(dX=H), INVALID),
    (dict(dW=A), INVALID), (dict(dW=B), INVALID), (dict(dW=C), INVALID), (dict(dW=D), INVALID), (dict(dW=H), INVALID),
    (dict(db=G), INVALID), (dict(db=A), INVALID), (dict(db=H + 64), INVALID), (dict(ws=A), INVALID), (dict(ws=D), INVALID),
])
def test_linear_grad_refusals(kw, expect):
    assert grad(**kw) == expect


def test_what_is_not_asked_for_is_not_needed():
    # refused for the output on its input, so after everything else was taken
    assert grad(dX=0, W=0, ldw=0, dW=A) == INVALID
    assert grad(dW=0, X=0, ldx=0, dX=A) == INVALID
    assert grad(act=0, Z=0, ldz=0, dX=A) == INVALID


def test_linear_workspace():
    need = sk.skinny_linear_grad_workspace(A, 48, B, 64, C, 64, 5, 48, 64, 1)
    assert grad(wsb=need - 1) == INVALID and need >= 5 * 96 * 2
    assert sk.skinny_linear_workspace(A, 64, B, 64, 5, 48, 64, 0) == 0
    for bad in ((-1, 48, 64, 1), (5, -1, 64, 1), (5, 48, MAX + 1, 1), (5, 48, 64, 7), (0, 48, 64, 1)):
        assert sk.skinny_linear_grad_workspace(A, 48, B, 64, C, 64, *bad) == 0
        assert sk.skinny_linear_workspace(A, 64, B, 64, *bad) == 0


def rotation(table=F, P=100, positions=F + (1 << 20), pair_axis=F + (1 << 21), axes=3, R=32, interleaved=0):
    return sk.skinny_rotation_t(table, P, positions, pair_axis, axes, R, interleaved)


def heads(q=A, qst=64 * 6, qsh=64, qw=C, Hq=4, k=A + 64 * 4 * 2, kst=64 * 6, ksh=64, kw=C + 4096, Hk=2, T=7, D=64, norm=1, dtype=0, qo=D,
          qost=256, qosh=64, ko=G, kost=128, kosh=64, rot=None, **r):
    return sk.skinny_qk_norm_rope(sk.skinny_heads_t(q, qst, qsh, qw, Hq), sk.skinny_heads_t(k, kst, ksh, kw, Hk),
                                  rot or rotation(**r), T, D, norm, 1e-6, dtype, qo, qost, qosh, ko, kost, kosh)


BAD_HEADS = [
    (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(D=513), UNSUPPORTED), (dict(axes=9), UNSUPPORTED), (dict(R=31), INVALID), (dict(R=66), INVALID), (dict(R=-2), INVALID),
    (dict(axes=0), INVALID), (dict(P=0), INVALID), (dict(table=0), INVALID), (dict(positions=0), INVALID),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(qsh=63), INVALID), (dict(qst=255), INVALID), (dict(qst=-384), INVALID),
    (dict(q=A + 1), MISALIGNED), (dict(k=A + 513), MISALIGNED), (dict(qw=C + 1), MISALIGNED), (dict(kw=C + 1), MISALIGNED),
    (dict(table=F + 2), MISALIGNED), (dict(positions=F + 2), MISALIGNED), (dict(pair_axis=F + 1), MISALIGNED),
    (dict(dtype=1, q=B + 2), MISALIGNED),
]


@pytest.mark.parametrize("kw,expect", BAD_HEADS + [
    (dict(T=0), sk.SKINNY_OK), (dict(Hq=0, Hk=0), sk.SKINNY_OK),
    (dict(qo=0), INVALID), (dict(ko=0), INVALID), (dict(qosh=63), INVALID), (dict(kost=127), INVALID), (dict(qo=D + 1), MISALIGNED),
    (dict(qo=A + 128, qost=384), INVALID), (dict(qo=A, qost=385), INVALID), (dict(ko=A, kost=384), INVALID),   # on inputs
    (dict(ko=D, kost=256), INVALID), (dict(ko=D + 512, kost=128), INVALID),                                   # on the other output
    (dict(qo=C), INVALID), (dict(qo=F), INVALID), (dict(ko=F + (1 << 20)), INVALID), (dict(ko=F + (1 << 21)), INVALID),
])
def test_heads_refusals(kw, expect):
    assert heads(**kw) == expect


def test_null_structures():
    lib = sk.load_library()
    q = sk.skinny_heads_t(A, 64, 64, 0, 1)
    null = ctypes.POINTER(sk.skinny_heads_t)()
    for a, b in ((null, q), (q, null)):
        assert lib.skinny_qk_norm_rope(a, b, rotation(), 1, 64, 1, 1e-6, 0, D, 64, 64, G, 64, 64, 0) == INVALID
    assert lib.skinny_qk_norm_rope(q, q, ctypes.POINTER(sk.skinny_rotation_t)(), 1, 64, 1, 1e-6, 0, D, 64, 64, G, 64, 64, 0) == INVALID


def heads_grad(dq=B, dqst=256, dqsh=64, dk=B + (1 << 20), dkst=128, dksh=64, q=A, qst=64 * 6, qsh=64, qw=C, Hq=4, k=A + 64 * 4 * 2,
               kst=64 * 6, ksh=64, kw=C + 4096, Hk=2, T=7, D=64, norm=1, dtype=0, qg=D, qgst=256, qgsh=64, kg=G, kgst=128, kgsh=64,
               qwg=H, kwg=H + 4096, ws=H + (1 << 20), wsb=1 << 20, **r):
    return sk.skinny_qk_norm_rope_grad(dq, dqst, dqsh, dk, dkst, dksh, sk.skinny_heads_t(q, qst, qsh, qw, Hq),
                                       sk.skinny_heads_t(k, kst, ksh, kw, Hk), rotation(**r), T, D, norm, 1e-6, dtype, qg, qgst,
                                       qgsh, kg, kgst, kgsh, qwg, kwg, ws, wsb)


@pytest.mark.parametrize("kw,expect", BAD_HEADS + [
    (dict(T=0, qwg=0, kwg=0), sk.SKINNY_OK), (dict(norm=0), INVALID), (dict(dq=0), INVALID), (dict(dk=0), INVALID), (dict(qg=0), INVALID),
    (dict(dqsh=63), INVALID), (dict(dkst=64), INVALID), (dict(kgsh=0), INVALID), (dict(dq=B + 1), MISALIGNED), (dict(kg=G + 1), MISALIGNED),
    (dict(qwg=H + 2), MISALIGNED), (dict(kwg=H + 4097), MISALIGNED), (dict(ws=0), INVALID), (dict(wsb=42 * 512 - 1), INVALID),
    (dict(ws=H + (1 << 20) + 8), MISALIGNED), (dict(qg=A, qgst=384), INVALID), (dict(qg=B + 64), INVALID), (dict(kg=B), INVALID),
    (dict(kg=D), INVALID), (dict(qg=H), INVALID), (dict(qg=H + (1 << 20)), INVALID), (dict(kwg=H), INVALID), (dict(qwg=A), INVALID),
    (dict(qwg=B), INVALID), (dict(kwg=C), INVALID), (dict(qwg=F), INVALID), (dict(ws=A), INVALID), (dict(ws=F), INVALID),
    (dict(ws=H), INVALID),
])
def test_heads_grad_refusals(kw, expect):
    assert heads_grad(**kw) == expect


def test_heads_workspace():
    assert sk.skinny_qk_norm_rope_grad_workspace(7, 4, 2, 64) == 42 * 2 * 64 * 4
    assert sk.skinny_qk_norm_rope_grad_workspace(1 << 20, 4, 2, 64) < 1 << 20
    for bad in ((-1, 4, 2, 64), (7, -1, 2, 64), (7, 4, -2, 64), (7, 4, 2, 0), (7, 4, 2, 513)):
        assert sk.skinny_qk_norm_rope_grad_workspace(*bad) == 0


def test_tensor_functions_refuse_what_they_cannot_take():
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sk.linear(x, x)                                  # not on a GPU
    with pytest.raises(ValueError):
        sk.linear_grad(x, x, x)
    with pytest.raises(ValueError):
        sk.qk_norm_rope(x.view(4, 2, 8), None)
    with pytest.raises(ValueError):
        sk.qk_norm_rope_grad(x.view(4, 2, 8), None, x.view(4, 2, 8), None)
