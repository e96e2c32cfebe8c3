"""Matrices of a product that share a buffer: refused where any element is shared, taken where none is (columns side
by side).  Pairs of small matrices are compared with the sets of their bytes.  No GPU needed, no kernel launched."""
import random

import pytest

import latency_skinny_bf16_gb300 as sk

BUF, FAR, SPACE = 0x7F0000000000, 0x7F1000000000, 0x7F2000000000      # fake, never dereferenced
TAKEN = (sk.SKINNY_OK, sk.SKINNY_ERR_NO_DEVICE, sk.SKINNY_ERR_LAUNCH)
INVALID = sk.SKINNY_ERR_INVALID_VALUE


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that no kernel may see")


def far(i):
    return FAR + (i << 24)


def linear(M, N, K, act=0, out=0, **at):
    """Every operand far from the others but those given as (address, row stride)."""
    rows = 2 * N if act in (1, 4) else N
    d = dict(X=(far(0), K), W=(far(1), K), R=(far(2), N), Y=(far(3), N), Z=(far(4), rows))
    d.update(at)
    return sk.skinny_linear_bf16(*d["X"], *d["W"], far(5), *d["R"], *d["Y"], *d["Z"], M, N, K, act, out, SPACE, 1 << 24)


def grad(M, N, K, **at):
    d = dict(dY=(far(0), N), X=(far(1), K), W=(far(2), K), Z=(far(3), N), dX=(far(4), K), dW=(far(5), K))
    d.update(at)
    return sk.skinny_linear_grad_bf16(*d["dY"], *d["X"], *d["W"], *d["Z"], *d["dX"], *d["dW"], far(6), M, N, K, 2, SPACE, 1 << 24)


def sizes(M, N, K, act=0, out=0):
    """Rows, columns and bytes of an element of each operand."""
    rows, ob = 2 * N if act in (1, 4) else N, 4 if out else 2
    return dict(X=(M, K, 2), W=(rows, K, 2), R=(M, N, ob), Y=(M, N, ob), Z=(M, rows, 2))


def bytes_of(at, ld, shape):
    r, c, el = shape
    return {at + (i * ld + j) * el + b for i in range(r) for j in range(c) for b in range(el)}


@pytest.mark.parametrize("M", [1, 2, 9])
@pytest.mark.parametrize("a,b", [("X", "Y"), ("Y", "X"), ("R", "Y"), ("Y", "R"), ("Y", "Z"), ("Z", "Y"), ("X", "Z"), ("R", "Z")])
def test_columns_side_by_side(a, b, M):
    N, K = 16, 24
    for act in (0, 1):
        size = sizes(M, N, K, act)
        ld = size[a][1] + size[b][1] + 8
        assert linear(M, N, K, act, **{a: (BUF, ld), b: (BUF + 2 * size[a][1], ld)}) in TAKEN
        assert linear(M, N, K, act, **{a: (BUF, ld), b: (BUF + 2 * size[a][1] - 2, ld)}) == INVALID
        if M > 1:      # one element of the next row
            assert linear(M, N, K, act, **{a: (BUF, size[a][1] + size[b][1] - 1), b: (BUF + 2 * size[a][1], size[a][1] + size[b][1] - 1)}) == INVALID


def test_columns_side_by_side_of_the_gradients():
    M, N, K = 5, 16, 24
    for a, b, wa in (("dY", "dX", N), ("dX", "dY", K), ("X", "dX", K), ("W", "dW", K), ("Z", "dX", N)):
        assert grad(M, N, K, **{a: (BUF, 64), b: (BUF + 2 * wa, 64)}) in TAKEN
        assert grad(M, N, K, **{a: (BUF, 64), b: (BUF + 2 * wa - 2, 64)}) == INVALID


def test_shared_elements_are_never_taken():
    rng = random.Random(7)
    shared = taken = 0
    for _ in range(8000):
        M, N, K, act, out = rng.choice([1, 2, 3]), rng.randrange(1, 6), rng.randrange(1, 6), rng.choice([0, 0, 1]), rng.choice([0, 1])
        size = sizes(M, N, K, act, out)
        a, b = rng.choice([("X", "Y"), ("Y", "Z"), ("R", "Y"), ("R", "Z"), ("X", "Z"), ("W", "Y"), ("W", "Z")])
        ld = rng.choice([8, 9, 12, 16])
        la, lb = (max(size[k][1], ld if rng.random() < 0.8 else rng.randrange(1, 16)) for k in (a, b))
        at = {a: (BUF, la), b: (BUF + 4 * rng.randrange(-20, 40) + (0 if out else 2 * rng.randrange(2)), lb)}
        if {a, b} == {"R", "Y"} and at["R"][0] == at["Y"][0] and (M == 1 or la == lb):
            continue                                   # the residual is the output
        status = linear(M, N, K, act, out, **at)
        if bytes_of(*at[a], size[a]) & bytes_of(*at[b], size[b]):
            assert status == INVALID, (M, N, K, act, out, at)
            shared += 1
        else:
            taken += status in TAKEN
    assert shared > 1500 and taken > 2000
