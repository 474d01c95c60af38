"""ts_verify_tree on the GPU: whole numbers, equal to the oracle's.

Where all values are multiples of 2^-k few enough to be added exactly (and the draft's mass is not divided by), kernel
and oracle are exact, so ties and borders are decided alike. Elsewhere the random numbers are 24-bit ones, and a
test or a running sum that the kernel holds to 2^-45 falls on the other side of one with a probability below 2^-20 a case.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draft_oracle as D
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _dev(x, t):
    return torch.as_tensor(np.asarray(x), dtype=t).to(DEV)


def _tree(n, rng, wide):
    return [-1] + [int(rng.integers(0, i)) if wide else int(rng.integers(max(0, i - 3), i)) for i in range(1, n)] if n else []


class Batch:
    def __init__(self, trees, V, seed=0, wide=True, make=None, extra=0, most=None):
        T = tsl()
        rng = np.random.default_rng(seed)
        self.trees, self.V = trees, V
        self.par = [_tree(n, rng, wide) for n in trees]
        rows = sum(trees) + extra
        self.cu = np.concatenate([[0], np.cumsum(trees)])
        if make is None:
            self.p, self.q = (rng.dirichlet(np.full(V, 0.3), size=rows).astype(np.float32) for _ in range(2))
        else:
            self.p, self.q = make(rng, rows, V)
        self.tok = np.zeros(rows, dtype=np.int64)
        for b, n in enumerate(trees):
            for i in range(1, n):
                w = np.maximum(self.q[self.cu[b] + self.par[b][i]].astype(np.float64), 0)
                self.tok[self.cu[b] + i] = rng.choice(V, p=w / w.sum()) if w.sum() > 0 else rng.integers(0, V)
        self.u, self.un = (rng.random(rows).astype(np.float32), rng.random(len(trees)).astype(np.float32))
        self.most = most or max(1, max(trees))
        self.ctx = T.Context(4, 4, 64, T.TS_KV_Q4, len(trees), 1, 1)

    def run(self, distinct, greedy, stream=None, pad=0):
        B = len(self.trees)
        path = torch.full((B, self.most), 99, dtype=torch.int32, device=DEV)
        count, nxt = (torch.full((B,), 99, dtype=torch.int32, device=DEV) for _ in range(2))
        par = [x for p in self.par for x in p] + [0] * (len(self.tok) - sum(self.trees))
        wide = [torch.full((len(self.tok), self.V + pad), float("nan"), device=DEV) for _ in range(2)]
        for w, x in zip(wide, (self.p, self.q)):
            w[:, :self.V] = _dev(x, torch.float32)
        p, q = (w[:, :self.V] for w in wide)
        self.ctx.verify_tree(_dev(self.tok, torch.int32), _dev(par, torch.int32), _dev(self.cu, torch.int32), p, None if greedy else q,
                             _dev(self.u, torch.float32), _dev(self.un, torch.float32), path, count, nxt, distinct, stream)
        torch.cuda.synchronize()
        return path.cpu().tolist(), count.cpu().tolist(), nxt.cpu().tolist()

    def check(self, number=float, pad=0, which=((False, False), (True, False), (False, True))):
        kept = 0
        for distinct, greedy in which:
            path, count, nxt = self.run(distinct, greedy, pad=pad)
            assert self.ctx.status() == 0
            for b, n in enumerate(self.trees):
                lo, hi = self.cu[b], self.cu[b + 1]
                if n == 0:
                    assert (path[b], count[b], nxt[b]) == ([-1] * self.most, 0, -1)
                    continue
                want, token = D.verify([int(x) for x in self.tok[lo:hi]], self.par[b], self.p[lo:hi], None if greedy else self.q[lo:hi],
                                       self.u[lo:hi], self.un[b], distinct, number)
                assert path[b] == want + [-1] * (self.most - len(want)), (b, distinct, greedy)
                assert count[b] == len(want) and nxt[b] == token, (b, distinct, greedy)
                kept += len(want)
        return kept


@pytest.mark.parametrize("V", [1, 2, 5, 31, 33, 500])
def test_small_vocabularies(V):
    b = Batch([1, 2, 0, 7, 16, 33, 9] * 4, V, seed=V, extra=2)
    assert b.check(pad=V % 3) > 28


@pytest.mark.parametrize("V", [2047, 2048, 4099, 9000, 32001])
def test_vocabularies_that_several_ctas_share(V):
    def near(rng, rows, V):
        z = rng.standard_normal((rows, V)) * 2
        out = []
        for x in (z, z + 0.7 * rng.standard_normal((rows, V))):
            e = np.exp(x - x.max(1, keepdims=True))
            out.append((e / e.sum(1, keepdims=True)).astype(np.float32))
        return out
    b = Batch([5, 1, 12], V, seed=V, wide=False, make=near)
    b.check(pad=1)


def test_the_largest_vocabulary():
    V = 1 << 20

    def make(rng, rows, V):
        p = np.full((rows, V), 2.0 ** -20, dtype=np.float32)
        q = np.zeros((rows, V), dtype=np.float32)
        q[:, V - 7] = 1.0
        return p, q
    b = Batch([2], V, make=make)
    b.un[:] = np.float32(1 - 2.0 ** -24)
    b.u[:] = 0.5
    path, count, nxt = b.run(False, False)
    # the drafted token is refused; of the others the last is drawn
    assert path[0] == [0, -1] and count == [1] and nxt == [V - 1]
    b.un[:] = 0.5                                                 # half of V - 1 tokens of equal mass: V / 2 - 1/2 of them
    assert b.run(False, False)[2] == [V // 2 - 1] and b.run(False, True)[2] == [V // 2 - 1]
    assert b.ctx.status() == 0


def _dyadic(rng, rows, V):
    """Probabilities that are multiples of 2^-10 and add up to one, many of them zero."""
    out = []
    for _ in range(2):
        x = np.zeros((rows, V))
        for r in range(rows):
            x[r] = rng.multinomial(1024, rng.dirichlet(np.full(V, 0.2)))
        out.append((x / 1024).astype(np.float32))
    return out


@pytest.mark.parametrize("V", [4, 40, 3001])
def test_borders_are_decided_exactly(V):
    """u of few bits, so that tests and running sums meet their borders; once with u = 0, once just below 1."""
    for seed in range(3):
        b = Batch([12, 3, 25, 1, 8], V, seed=seed, make=_dyadic)
        rng = np.random.default_rng(seed)
        which = ((False, False), (False, True))
        for u in (rng.integers(0, 16, len(b.u)) / 16, np.zeros(len(b.u)), np.full(len(b.u), 1 - 2.0 ** -24)):
            b.u = u.astype(np.float32)
            for un in (rng.integers(0, 1024, 5) / 1024, np.zeros(5), np.full(5, 1 - 2.0 ** -24)):
                b.un = un.astype(np.float32)
                b.check(Fraction, which=which)


def test_equal_distributions_keep_every_draft():
    b = Batch([20, 6], 300, seed=4, wide=False)
    b.q = b.p.copy()
    for b_, n in enumerate(b.trees):
        b.par[b_] = [-1] + list(range(n - 1))
        for i in range(1, n):
            b.tok[b.cu[b_] + i] = int(np.argmax(b.p[b.cu[b_] + i - 1]))
    path, count, nxt = b.run(False, False)
    assert count == [20, 6] and path[0] == list(range(20))
    # refused although p = q (u is 1): nothing is left, the token comes from p itself
    b.u[:] = 1.0
    b.check(which=((False, False),))


def test_entries_that_are_no_number_count_as_zero():
    def make(rng, rows, V):
        p, q = _dyadic(rng, rows, V)
        p[:, 3] = np.nan
        p[:, 5], q[:, 6] = -0.5, -0.25
        q[:, 4] = 0
        return p, q
    b = Batch([9, 1, 17], 40, seed=6, make=make)
    b.q = np.maximum(b.q, 0)
    b.check(Fraction, which=((False, False), (False, True)))
    q = b.q.copy()
    b.q[:, 4], b.q[:, 6] = np.where(q[:, 4] == 0, np.nan, q[:, 4]), np.where(q[:, 6] == 0, -1.0, q[:, 6])
    b.check(Fraction, which=((False, False),))
    b.p[:] = np.nan
    path, count, nxt = b.run(False, False)
    assert count == [1, 1, 1] and nxt == [-1, -1, -1] and b.ctx.status() == 0


def test_the_longest_tree():
    """1024 nodes: a chain that is kept to its end, and a root with 1023 children: the first is taken (u q is below p), or, as
    drafts without probabilities and u = 1, none."""
    V, n = 2000, 1024
    for greedy in (False, True):
        b = Batch([n, n], V, seed=7, make=lambda rng, rows, V: (np.full((rows, V), 1.0 / 2048, dtype=np.float32),) * 2)
        b.par = [[-1] + list(range(n - 1)), [-1] + [0] * (n - 1)]
        b.tok[:] = np.tile(np.arange(n), 2)
        b.u[:n], b.u[n:] = 0.0, 1.0
        if not greedy:
            b.q = np.full((2 * n, V), 1.0 / 4096, dtype=np.float32)
        b.un[:] = 0.25
        path, count, nxt = b.run(False, greedy)
        assert path[0] == list(range(n)) and nxt[0] == V // 4
        lo = slice(n, 2 * n)
        want, token = D.verify(list(range(n)), b.par[1], b.p[lo], None if greedy else b.q[lo], b.u[lo], b.un[1], False)
        assert want == ([0] if greedy else [0, 1])
        assert path[1] == want + [-1] * (n - len(want)) and count == [n, len(want)] and nxt[1] == token and b.ctx.status() == 0


def test_a_thousand_refusals():
    """The drafter's mass lies on 1024 tokens, twice what the target gives them: every child is refused, whatever is summed
    in between, and the token comes from the others."""
    V, n = 2000, 1024

    def make(rng, rows, V):
        p, q = np.full((rows, V), 1.0 / 2048, dtype=np.float32), np.zeros((rows, V), dtype=np.float32)
        q[:, :n] = 1.0 / 1024
        return p, q
    b = Batch([n], V, seed=8, make=make)
    b.par = [[-1] + [0] * (n - 1)]
    b.u[:] = 1.0
    for un, token in ((0.0, n), (0.5, n + (V - n) // 2), (1 - 2.0 ** -24, V - 1)):
        b.un[:] = un
        for distinct in (False, True):
            path, count, nxt = b.run(distinct, False)
            assert path[0] == [0] + [-1] * (n - 1) and count == [1] and nxt == [token] and b.ctx.status() == 0


def test_errors_are_recorded():
    T = tsl()
    # a node of a bad token and one of a bad parent: passed over, with their subtrees
    b = Batch([8, 4], 50, seed=8, wide=False)
    b.tok[2], b.par[0][5], b.tok[9] = 50, 6, -1
    got = b.run(False, False)
    assert b.ctx.status() == T.STATUS_CODE["TS_ERR_INVALID_ARG"]
    for s in (0, 1):
        lo, hi = b.cu[s], b.cu[s + 1]
        want, token = D.verify([int(x) for x in b.tok[lo:hi]], b.par[s], b.p[lo:hi], b.q[lo:hi], b.u[lo:hi], b.un[s], False)
        assert got[0][s][:len(want)] == want and got[1][s] == len(want) and got[2][s] == token
    # a path that does not fit
    b = Batch([20, 6], 30, seed=4, wide=False, most=3)
    b.q, b.u[:] = b.p.copy(), 0.0
    b.par = [[-1] + list(range(19)), [-1] + list(range(5))]
    b.tok[:] = [int(np.argmax(b.p[max(0, r - 1)])) for r in range(26)]
    path, count, nxt = b.run(False, False)
    assert b.ctx.status() == T.STATUS_CODE["TS_ERR_CAPACITY"] and path[0] == [0, 1, 2] and count == [20, 6]
    # boundaries, and more nodes than a sequence may have
    for cu in ([0, 30, 26], [1, 20, 26], [0, 20, 1000], [0, -3, 26]):
        b.cu = np.array(cu)
        path, count, nxt = b.run(False, False)
        assert b.ctx.status() == T.STATUS_CODE["TS_ERR_SEQ_LEN"]
        bad = [s for s in (0, 1) if not (0 <= cu[s] <= cu[s + 1] <= 26 and (s or cu[0] == 0))]
        assert bad and all(count[s] == 0 and nxt[s] == -1 and path[s] == [-1] * 3 for s in bad)
    b = Batch([1025], 4, seed=9)
    assert b.run(False, False)[1] == [0] and b.ctx.status() == T.STATUS_CODE["TS_ERR_SEQ_LEN"]


def test_captured_and_replayed():
    b = Batch([9, 30, 2], 700, seed=10)
    want = b.run(True, False)
    args = [_dev(b.tok, torch.int32), _dev([x for p in b.par for x in p], torch.int32), _dev(b.cu, torch.int32),
            _dev(b.p, torch.float32), _dev(b.q, torch.float32), _dev(b.u, torch.float32), _dev(b.un, torch.float32)]
    path, count, nxt = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((3, 30), (3,), (3,)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.ctx.verify_tree(*args, path, count, nxt, True)
    for _ in range(2):
        path.fill_(5)
        g.replay()
        assert (path.cpu().tolist(), count.cpu().tolist(), nxt.cpu().tolist()) == want


@pytest.mark.parametrize("distinct,greedy", [(False, False), (True, False), (False, True)])
def test_tokens_come_out_as_the_target_has_them(distinct, greedy):
    """4096 roots with three drafts each, of one target: the token behind the root is distributed as the target."""
    V, B, n = 6, 4096, 4
    rng = np.random.default_rng(11)
    p, q = rng.dirichlet(np.ones(V), 2).astype(np.float32)
    b = Batch([n] * B, V, seed=12, make=lambda rng, rows, V: (np.tile(p, (rows, 1)), np.tile(q, (rows, 1))))
    for s in range(B):
        b.par[s] = [-1, 0, 0, 0]
        if distinct or greedy:
            b.tok[4 * s + 1:4 * s + 4] = rng.choice(V, 3, replace=False, p=q.astype(np.float64) / q.sum(dtype=np.float64))
    path, count, nxt = b.run(distinct, greedy)
    first = [int(b.tok[4 * s + path[s][1]]) if count[s] > 1 else nxt[s] for s in range(B)]
    seen = np.bincount(first, minlength=V) / B
    # five standard deviations of a share of 4096
    assert np.all(np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / B) + 1e-3)
