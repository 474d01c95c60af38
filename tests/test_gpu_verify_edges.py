"""ts_verify_tree on the GPU where a walk ends at once, and at the edges of its arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import draft_oracle as D
from parity import tsl
from test_gpu_verify import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [40, 5000, 20000])
def test_walks_that_end_at_once(V):
    """Sequences without rows and with bad boundaries reach the first message to the other CTAs of their cluster at once:
    hundreds of them, among others that draw a token, call behind call."""
    trees = [0 if b % 5 else 1 for b in range(400)]
    rows = sum(trees)

    def make(rng, n, V):
        p = np.zeros((n, V), dtype=np.float32)
        p[np.arange(n), (np.arange(n) * 977) % V] = 1.0
        return p, p
    b = Batch(trees, V, seed=V, make=make)
    want = [-1 if b_ % 5 else ((b_ // 5) * 977) % V for b_ in range(400)]
    for _ in range(5):
        path, count, nxt = b.run(False, False)
        assert nxt == want and count == trees and [p[0] for p in path] == [t - 1 for t in trees]
    assert b.ctx.status() == 0
    cu = b.cu.copy()
    b.cu = np.where(np.arange(401) % 2 == 1, rows + 5, b.cu)      # every sequence ends or begins beyond the rows
    path, count, nxt = b.run(False, False)
    assert set(nxt) == {-1} and set(count) == {0} and b.ctx.status() == tsl().STATUS_CODE["TS_ERR_SEQ_LEN"]
    b.cu = cu
    assert b.run(False, False)[2] == want and b.ctx.status() == 0


def _border(seed, V):
    """A node with three children whose third is decided by a small sum of small residuals: half of the draft's mass lies
    on tokens that the target gives a little less, the other half on ones that it gives a little more. The first two
    children are of the former (refused at u just below 1), and c = 1 + Z of the second test has 24 bits and more.
    Returns p, q, the tokens and the smallest u at which the third child is refused, by exact arithmetic."""
    rng = np.random.default_rng(seed)
    few = np.arange(V // 2)
    q = np.concatenate([rng.uniform(0.5, 1, V // 2), rng.uniform(0.5, 1, V - V // 2)])
    q[few] *= 0.5 / q[few].sum()
    q[V // 2:] *= 0.5 / q[V // 2:].sum()
    eps = 2.0 ** -9
    p = q.copy()
    p[few] *= 1 - 2 * eps
    p[V // 2:] *= 1 + 2 * eps * rng.uniform(0.6, 1.4, V - V // 2)
    p, q = p.astype(np.float32), q.astype(np.float32)
    P, Q = [Fraction(float(x)) for x in p], [Fraction(float(x)) for x in q]
    c = 1 + sum(max(a - b, 0) for a, b in zip(P, Q))
    Z = sum(max(a - c * b, 0) for a, b in zip(P, Q))
    for x in range(V // 2, V):
        u = max(P[x] - c * Q[x], 0) / (Q[x] * Z)
        if Fraction(1, 8) < u < Fraction(15, 16):
            break
    else:
        return None
    lo = np.float32(float(u))
    if Fraction(float(lo)) >= u:
        lo = np.nextafter(lo, np.float32(0))
    hi = np.nextafter(lo, np.float32(1))
    # (the kernel's sum is right to 2^-40 of it: borders that near to a number that u can take are left to others)
    if min(u - Fraction(float(lo)), Fraction(float(hi)) - u) < u / 2 ** 38:
        return None
    return p, q, [0, 0, 1, x], lo, hi


@pytest.mark.parametrize("V", [8, 62])
def test_small_residuals_are_summed_as_exact_arithmetic_does(V):
    """u just below and at the border of a test against a sum of p - c q that is a thousandth of p and q: products that were
    rounded once in one place and not in another would be 2^-15 off, u is told apart by 2^-24."""
    cases = [c for c in (_border(seed, V) for seed in range(60)) if c is not None]
    assert len(cases) >= 20
    B = 2 * len(cases)
    b = Batch([4] * B, V, make=lambda rng, rows, V: (np.zeros((rows, V), dtype=np.float32), np.ones((rows, V), dtype=np.float32)))
    for s in range(B):
        p, q, tokens, lo, hi = cases[s // 2]
        rows = slice(4 * s, 4 * s + 4)
        b.par[s], b.p[rows], b.q[rows], b.tok[rows] = [-1, 0, 0, 0], p, q, tokens
        b.u[rows] = [0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, hi if s % 2 else lo]
    path, count, nxt = b.run(False, False)
    assert b.ctx.status() == 0
    for s in range(B):
        want, _ = D.verify(list(b.tok[4 * s:4 * s + 4]), b.par[s], b.p[4 * s:4 * s + 4], b.q[4 * s:4 * s + 4], b.u[4 * s:4 * s + 4],
                           b.un[s], False, Fraction)
        assert want == ([0] if s % 2 else [0, 3])
        assert path[s][:count[s]] == want, s


@pytest.mark.parametrize("V", [7, 40, 2047, 9000, 32001, 128256])
def test_a_number_that_rounds_to_one_draws_the_last_token(V):
    """u_next of 1 (a number from [0, 1) of more bits, rounded): no running sum passes it, so the last token that has mass."""
    rng = np.random.default_rng(V)
    B = 6

    def make(rng, rows, V):
        p = np.full((rows, V), 1.0 / V, dtype=np.float32)
        for r, last in enumerate([V - 1, V // 2, 0, V - 2, V // 3, 3 * V // 4]):
            p[r, last + 1:] = 0.0
        return p, p
    b = Batch([1] * B, V, make=make)
    last = [V - 1, V // 2, 0, V - 2, V // 3, 3 * V // 4]
    b.un[:] = 1.0
    for distinct, greedy in ((False, False), (True, False), (False, True)):
        path, count, nxt = b.run(distinct, greedy)
        assert nxt == last and count == [1] * B
    b.un[:] = rng.random(B)
    b.un[0] = 1 - 2.0 ** -24
    assert b.run(False, False)[2][0] == V - 1
    b.check(which=((False, False),))
