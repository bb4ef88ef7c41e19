"""draft_verify where what a fall leaves of a token is small beside the token's probabilities,
against the rule in rational numbers."""

from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest

import tree_ref as ref
from test_gpu_draft_verify import check, gb, run  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def want_of(p, q, tokens, parents, u):
    S, Tn, V = p.shape
    return [ref.verify_exact(p[r].tolist(), None if q is None else q[r].tolist(), tokens[r], parents[r],
                             np.asarray(u[r], dtype=np.float32).tolist(), Tn, V) for r in range(S)]


def test_a_remainder_below_the_rounding_of_its_product(gb):
    """Both children fall; what is left is 2.3e-8 on token 1 alone, where the product in fp32
    rounds past p."""
    p = np.tile(np.float32([float.fromhex("0x1.944ea0p-4"), float.fromhex("0x1.cd762cp-1"), 0]), (1, 3, 1))
    q = np.tile(np.float32([float.fromhex("0x1.9442p-4"), float.fromhex("0x1.cd67cp-1"), 2.0 ** -13]), (1, 3, 1))
    tokens, parents, u = np.array([[0, 2, 2]]), np.array([[-1, 0, 0]]), [[0.05, 0.5, 0.5]]
    want = want_of(p, q, tokens, parents, u)
    assert want == [([1], [0])]
    check(run(gb, p, q, tokens, parents, u), want, 3)


@pytest.mark.parametrize("S,V", [(500, 3), (40, 4099)])
def test_remainders_next_to_nothing(gb, S, V):
    """Rows that sum to 1 in steps of 2^-24, with p = q (1 + 2^-13) but for less than a step:
    the first fall leaves W = 2^-13, the second rem and 1/4 - rem steps on two tokens, or one of
    them on one token.  The kernel's sums are off by less than 2^-43 a token, 2^-17 of the 2^-26
    that is left."""
    rng = np.random.default_rng(V)
    p, q = np.zeros((2, S, 3, V), dtype=np.float32)
    tokens = np.zeros((S, 3), dtype=np.int64)
    u = np.full((S, 3), 0.5)
    for r in range(S):
        x, y, z = rng.choice(V, 3, replace=False)
        a = int(rng.integers(1 << 16, (1 << 24) - (1 << 16)))
        up = a * (1 + 2.0 ** -13)  # (exact)
        b = int(np.floor(up)) + int(rng.integers(0, 2))
        rem = b - up
        q[r, :, [x, y, z]] = np.array([[a], [(1 << 24) - a - (1 << 11)], [1 << 11]]) * 2.0 ** -24
        p[r, :, [x, y]] = np.array([[b], [(1 << 24) - b]]) * 2.0 ** -24
        tokens[r] = z
        border = (rem if x < y else 0.25 - rem) / 0.25  # between the two tokens, if in (0, 1)
        u[r, 0] = max((0.25, 0.5, 0.75), key=lambda v: abs(v - border))
    parents = np.tile([-1, 0, 0], (S, 1))
    assert all(Fraction(float(s)) == 1 for s in p[:, 0].astype(np.float64).sum(-1))
    check(run(gb, p, q, tokens, parents, u), want_of(p, q, tokens, parents, u), 3)


@pytest.mark.parametrize("n", [130, 180, 256])
def test_many_falls_over_rows_that_sum_to_almost_4(gb, n):
    """What the siblings have taken off comes to A = 1 + 3.9 a fall or so, to 446, 595 and 799."""
    S, V = 64, 5
    p = np.tile(np.float32([1, 1, 1, 0.875, 0]), (S, n, 1))
    q = np.tile(np.float32([2.0 ** -10, 2.0 ** -12, 2.0 ** -11, 0, 2.0 ** -20]), (S, n, 1))
    tokens, parents = np.full((S, n), 4), np.tile([-1] + [0] * (n - 1), (S, 1))
    u = np.full((S, n), 0.5)
    u[:, 0] = (np.arange(S) + 0.5) / S
    want = ref.verify_exact(p[0].tolist(), q[0].tolist(), tokens[0], parents[0], u[0].tolist(), n, V)
    # (requests differ in the last draw alone: the falls are those of the first request)
    w, W, A = [Fraction(float(x)) for x in p[0, 0]], Fraction(1), Fraction(0)
    row = [Fraction(float(x)) for x in q[0, 0]]
    for _ in range(n - 1):
        A += W
        w = [max(Fraction(float(a)) - A * b, Fraction(0)) for a, b in zip(p[0, 0], row)]
        W = sum(w)
    runs = np.cumsum([float(x) for x in w]) / float(W)
    assert np.abs(runs[:, None] - u[:, 0]).min() > 2.0 ** -20  # no number next to a border
    tokens_last = [int(np.searchsorted(runs, x, side="right")) for x in u[:, 0]]
    assert tokens_last[0] == want[0][0] and (n < 180 or A > 512)
    check(run(gb, p, q, tokens, parents, u), [([x], [0]) for x in tokens_last], n)


def test_a_token_that_fell_falls_again_however_small(gb):
    """Without a draft: a token below the sums' step is gone all the same once it has fallen."""
    S, V = 4, 6
    tokens = np.array([[0, 1, 1], [0, 5, 5], [0, 3, 3], [0, 0, 0]])
    parents = np.tile([-1, 0, 0], (S, 1))
    p = np.zeros((S, 3, V), dtype=np.float32)
    p[:3, :, 0], p[3, :, 1] = 1, 1
    for r, small in enumerate((2.0 ** -50, 2.0 ** -46, 2.0 ** -60, 2.0 ** -49)):
        p[r, :, tokens[r, 1]] = small
    u = np.tile([0.5, 0.25, 0.0], (S, 1))
    want = want_of(p, None, tokens, parents, u)
    assert all(path == [0] for _, path in want)
    check(run(gb, p, None, tokens, parents, u), want, 3)


@pytest.mark.parametrize("small", [2.0 ** -33, 2.0 ** -35, 2.0 ** -38])
def test_a_child_of_nothing_falls(gb, small):
    """p is below q by a step of 2^-56 and less at the fallen token: nothing is left there, and a
    second child of it falls even for the number 0."""
    step = small * 2.0 ** -23
    p = np.tile(np.float32([small + step, 0.75, 0.25]), (1, 3, 1))
    q = np.tile(np.float32([small + 2 * step, 0.25, 0.75]), (1, 3, 1))
    tokens, parents, u = np.array([[0, 0, 0]]), np.array([[-1, 0, 0]]), [[0.5, 1 - 2.0 ** -24, 0.0]]
    want = want_of(p, q, tokens, parents, u)
    assert want == [([1], [0])]
    check(run(gb, p, q, tokens, parents, u), want, 3)
