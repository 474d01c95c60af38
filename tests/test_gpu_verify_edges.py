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
