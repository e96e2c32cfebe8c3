"""Outputs of the heads' operators that share a buffer: refused where any element is shared, taken where none is.
Every pair of small views is compared with the sets of their elements.  No GPU needed, no kernel launched."""
import itertools
import random

import pytest

import latency_skinny_bf16_gb300 as sk

BUF, FAR = 0x7F0000000000, 0x7F1000000000      # fake, never dereferenced
TAKEN = (sk.SKINNY_OK, sk.SKINNY_ERR_NO_DEVICE, sk.SKINNY_ERR_LAUNCH)
INVALID = sk.SKINNY_ERR_INVALID_VALUE


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that no kernel may see")


def call(q, k, T, D):
    """Outputs at (element offset, token stride, head stride, heads) of one buffer, the inputs elsewhere."""
    heads = [sk.skinny_heads_t(FAR + (i << 24), 1 << 10, D, 0, v[3]) for i, v in enumerate((q, k))]
    rot = sk.skinny_rotation_t(0, 1, 0, 0, 1, 0, 0)
    (qo, qst, qsh, _), (ko, kst, ksh, _) = q, k
    return sk.skinny_qk_norm_rope(*heads, rot, T, D, 1, 1e-6, 0, BUF + 2 * qo, qst, qsh, BUF + 2 * ko, kst, ksh)


def elements(v, T, D):
    return {v[0] + t * v[1] + h * v[2] + d for t in range(T) for h in range(v[3]) for d in range(D)}


@pytest.mark.parametrize("T", [1, 2, 7])
@pytest.mark.parametrize("order", ["by turns", "heads first by turns", "one key", "groups"])
def test_heads_by_turns_are_taken(order, T):
    """[T, H, 3, D], queries, keys and values of a head beside each other, and their like: in place or elsewhere."""
    H, D = 4, 8
    q, k = {
        "by turns": ((0, H * 3 * D, 3 * D, H), (D, H * 3 * D, 3 * D, H)),
        "heads first by turns": ((0, 3 * D, T * 3 * D, H), (D, 3 * D, T * 3 * D, H)),
        "one key": ((0, (H + 2) * 2 * D, 2 * D, H), (D, (H + 2) * 2 * D, 2 * D, 1)),
        "groups": ((0, 2 * H * 3 * D, 3 * D, 2 * H), (D, 2 * H * 3 * D, 6 * D, H)),
    }[order]
    assert not elements(q, T, D) & elements(k, T, D)
    assert call(q, k, T, D) in TAKEN
    # in place
    hq, hk = (sk.skinny_heads_t(BUF + 2 * v[0], v[1], v[2], 0, v[3]) for v in (q, k))
    rot = sk.skinny_rotation_t(0, 1, 0, 0, 1, 0, 0)
    assert sk.skinny_qk_norm_rope(hq, hk, rot, T, D, 1, 1e-6, 0, hq.x, q[1], q[2], hk.x, k[1], k[2]) in TAKEN
    # gradients in place of dq and dk
    x = [sk.skinny_heads_t(FAR + (i << 24), v[3] * D, D, 0, v[3]) for i, v in enumerate((q, k))]
    assert sk.skinny_qk_norm_rope_grad(hq.x, q[1], q[2], hk.x, k[1], k[2], *x, rot, T, D, 1, 1e-6, 0, hq.x, q[1], q[2], hk.x, k[1],
                                       k[2], 0, 0, 0, 0) in TAKEN


def test_shared_elements_are_never_taken():
    rng = random.Random(5)
    taken = shared = 0
    for _ in range(6000):
        T, D = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4])
        views = []
        for _ in range(2):
            H = rng.choice([1, 2, 3])
            inner = D * rng.choice([1, 2, 3]) + rng.choice([0, 0, 0, 1])
            outer = inner * rng.choice([1, 2, 3, 4, 6]) + rng.choice([0, 0, 0, 1, 2])
            st, sh = (outer, inner) if rng.random() < 0.7 else (inner, outer)
            views.append((rng.randrange(0, 24), st, sh, H))
        if any(len(elements(v, T, D)) < T * v[3] * D for v in views):
            continue
        status = call(*views, T, D)
        if elements(views[0], T, D) & elements(views[1], T, D):
            assert status == INVALID, (views, T, D)
            shared += 1
        else:
            taken += status in TAKEN
    assert shared > 500 and taken > 500
