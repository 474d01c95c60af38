"""ts_verify_tree on the GPU where a walk ends at once, and at the edges of its arithmetic."""
import numpy as np
import pytest

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
