"""ts_tree_attend on the GPU against the fp64 oracle: trees of drafts over a paged cache, causal drafts, masks that
leave rows empty, odd lengths and pages, and hidden places that hold NaN or infinities.

Tolerance, per row with weights w and values v, as for the prompt attention: a score is a sum of d products that are exact in
fp32, off by el = alpha sum|q_e k_e| (d + 16) 2^-24, and its exponential by 2^-20; a weight is rounded to bf16 for its
product (2^-8), sums of n terms are off by n 2^-23, each of at most 8 parts is scaled once more (2^-20), the output is rounded to bf16
(2^-8).
"""
import math

import numpy as np
import pytest
import torch

from oracle import draft_oracle as D
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
GEOS = [(8, 4, 128), (4, 7, 128), (8, 1, 128), (4, 2, 64), (2, 8, 128)]


class Case:
    """Pools whose pages are scattered, every slot that no token has filled with NaN; trees; masks of their ancestors."""

    def __init__(self, HKV, G, d, lens, trees, page=16, seed=0, spread=1.5, extra=0, mask="tree", spare=0):
        T = tsl()
        self.T, self.HKV, self.G, self.d, self.page = T, HKV, G, d, page
        self.lens, self.trees, self.B, self.H = lens, trees, len(lens), HKV * G
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        np_ = [(n + page - 1) // page for n in lens]
        self.pages = max(1, sum(np_)) + spare
        max_pages = max(1, max(np_))
        perm = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((self.B, max_pages), -7, dtype=np.int32)          # (entries past a sequence are unused)
        at = 0
        self.k_pool, self.v_pool = (torch.full((self.pages, HKV, page, d), float("nan"), dtype=BF, device=DEV) for _ in range(2))
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            self.table[b, :np_[b]] = perm[at:at + np_[b]]
            at += np_[b]
            k, v = (torch.randn(n, HKV, d, generator=g, device=DEV).to(BF) for _ in range(2))
            pos = torch.arange(n, device=DEV)
            p = torch.from_numpy(self.table[b]).to(DEV).long()[pos // page]
            self.k_pool[p, :, pos % page], self.v_pool[p, :, pos % page] = k, v
            self.k.append(k)
            self.v.append(v)
        self.cu = np.concatenate([[0], np.cumsum(trees)]).astype(np.int32)
        rows = int(self.cu[-1]) + extra
        m = torch.randn(rows, self.H * d + 8, generator=g, device=DEV) * spread
        self.q = m.to(BF)[:, :self.H * d].view(rows, self.H, d)
        self.words = max(1, (max(trees) + 31) // 32)
        self.bits = None
        if mask is not None:
            self.bits = []
            for t in trees:
                anc = []
                for i in range(t):
                    if mask == "tree":
                        p = int(rng.integers(max(0, i - 5), i)) if i else -1
                        anc.append((anc[p] if p >= 0 else 0) | 1 << i)
                    else:
                        anc.append(mask(t, i, rng))
                self.bits += anc
        self.out = torch.full((rows, self.H, d), 7.0, dtype=BF, device=DEV)
        self.lse = torch.full((rows, self.H), 7.0, device=DEV)
        self.ctx = T.Context(self.H, HKV, d, T.TS_KV_BF16, self.B, max_pages, self.pages, page)

    def dev(self, x):
        return torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV)

    def mask_tensor(self):
        if self.bits is None:
            return None
        m = np.zeros((self.q.shape[0], self.words), dtype=np.uint32)
        for r, x in enumerate(self.bits):
            for w in range(self.words):
                m[r, w] = x >> (32 * w) & 0xffffffff
        return torch.from_numpy(m.view(np.int32)).to(DEV)

    def run(self, scale=0.0, stream=None, lens=None, table=None, cu=None):
        self.ctx.tree_attend(self.q, self.k_pool, self.v_pool, self.dev(self.table if table is None else table),
                             self.dev(self.lens if lens is None else lens), self.dev(self.cu if cu is None else cu),
                             self.mask_tensor(), self.out, self.lse, scale, stream)
        return self

    def check(self, scale=None, rows=None, heads=None, hidden=None):
        """hidden: {sequence: positions that nobody sees}"""
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        q, out, lse = (x.double().cpu().numpy() for x in (self.q, self.out, self.lse))
        worst = 0.0
        for b, (n, t) in enumerate(zip(self.lens, self.trees)):
            k, v = self.k[b].double().cpu().numpy(), self.v[b].double().cpu().numpy()
            for i in range(t) if rows is None else [x for x in rows if x < t]:
                r = int(self.cu[b]) + i
                seen = D.tree_seen(n, t, i, None if self.bits is None else self.bits[r])
                if hidden and b in hidden:
                    seen[hidden[b]] = False
                for h in range(self.H) if heads is None else heads:
                    kk, vv = k[:, h // self.G], v[:, h // self.G]
                    want, wl, w = D.tree_attend(q[r, h], kk, vv, seen, scale)
                    if not seen.any():
                        assert np.all(out[r, h] == 0) and lse[r, h] == -math.inf
                        continue
                    el = abs(scale) * float(np.max(np.abs(kk[seen]) @ np.abs(q[r, h]))) * (self.d + 16) * 2.0 ** -24
                    tol = (w[seen] @ np.abs(vv[seen])) * (2.0 ** -8 + 2 * el + 9 * 2.0 ** -20 + n * 2.0 ** -23) + np.abs(want) * 2.0 ** -8
                    off = np.abs(out[r, h] - want)
                    worst = max(worst, float(np.max(off / (tol + 1e-30))))
                    assert np.all(off <= tol + 1e-30), (b, i, h, worst)
                    assert abs(lse[r, h] - wl) <= el + n * 2.0 ** -23 + 9 * 2.0 ** -20 + abs(wl) * 2.0 ** -22, (b, i, h, lse[r, h], wl)
        assert self.ctx.status() == 0
        return worst


@pytest.mark.parametrize("HKV,G,d", GEOS)
def test_small_trees(HKV, G, d):
    c = Case(HKV, G, d, lens=[1, 17, 128, 300, 5, 129], trees=[1, 5, 3, 16, 5, 0], extra=3)
    c.run().check()
    assert torch.all(c.out[int(c.cu[-1]):] == 7.0) and torch.all(c.lse[int(c.cu[-1]):] == 7.0)


@pytest.mark.parametrize("HKV,G,d", GEOS)
def test_drafts_up_to_their_own(HKV, G, d):
    Case(HKV, G, d, lens=[1, 40, 700, 257], trees=[1, 40, 33, 130], mask=None, seed=1).run().check(heads=[0, HKV * G - 1])


@pytest.mark.parametrize("HKV,G,d,trees", [(8, 4, 128, [64, 65, 33]), (4, 7, 128, [36, 37, 19]), (8, 1, 128, [256, 257, 129]),
                                           (4, 2, 64, [128, 129, 65]), (2, 8, 128, [32, 33, 200])])
def test_blocks_of_one_and_two_tiles(HKV, G, d, trees):
    """Trees that fill a tile, two tiles, and one more token; several key tiles, shares that begin inside blocks."""
    Case(HKV, G, d, lens=[2000, 1500, 900], trees=trees, seed=2).run().check(rows=[0, 1, 17, 18, 31, 32, 63, 64, 127, 128, 256, 199],
                                                                            heads=[0, G - 1, HKV * G - 1])


@pytest.mark.parametrize("n", [16, 127, 128, 129, 255, 256, 257, 383, 1000, 20000])
def test_lengths_around_tiles(n):
    """One sequence over all SMs: every KV head's key tiles are shared out, parts joined."""
    Case(8, 4, 128, lens=[n], trees=[9], seed=n).run().check(heads=[0, 5, 31])


@pytest.mark.parametrize("trees", [[5, 33, 18, 19, 1, 36, 0, 24], [33, 5, 19, 2, 40, 17, 36, 1]])
def test_shares_over_blocks_of_one_and_two_tiles(trees):
    """CTAs whose shares go from long blocks of one tile to blocks of two and back."""
    Case(4, 7, 128, lens=[20000, 19000, 20011, 18001, 20000, 17000, 300, 20001], trees=trees, seed=19).run().check(rows=[0, 17, 18, 35], heads=[0, 27])


def test_thousand_drafts():
    def some(t, i, rng):
        return int.from_bytes(rng.bytes(t // 8), "little")
    c = Case(8, 4, 128, lens=[1024, 1500], trees=[1024, 1000], mask=some, seed=3)
    c.run().check(rows=[0, 1, 500, 511, 512, 999, 1023], heads=[0, 13, 31])


def test_masks_of_any_bits_and_empty_rows():
    """Rows that see nothing give zeros and -inf: no prefix and no bit, in one part of a block or in all."""
    def odd(t, i, rng):
        return [0, 1 << i, (1 << t) - 1, 0xaaaaaaaaaa & ((1 << t) - 1), 1 << (t - 1)][i % 5]
    Case(8, 4, 128, lens=[40, 12, 300], trees=[40, 12, 40], mask=odd, seed=4).run().check(heads=[0, 31])
    # a prefix of 130 tokens that no row's own scores outweigh
    Case(4, 2, 64, lens=[170], trees=[40], mask=lambda t, i, rng: 0, seed=5).run().check()


def test_many_sequences():
    rng = np.random.default_rng(0)
    trees = [int(x) for x in rng.integers(0, 20, 70)]
    lens = [t + int(rng.integers(0, 400)) for t in trees]
    Case(4, 2, 64, lens=lens, trees=trees, seed=6).run().check(heads=[0, 3, 7])


def test_hundreds_of_sequences():
    """More sequences than the look-ups take at a time; most blocks whole, some split."""
    rng = np.random.default_rng(1)
    trees = [int(x) for x in rng.integers(0, 5, 230)]
    trees[200] = 100
    lens = [t + int(rng.integers(0, 60)) for t in trees]
    lens[35], lens[200], lens[229] = trees[35] + 5000, 3000, trees[229] + 2000
    Case(4, 2, 64, lens=lens, trees=trees, seed=20).run().check(rows=[0, 3, 99], heads=[0, 7])


def test_one_token_pages():
    Case(8, 1, 128, lens=[1, 260, 129], trees=[1, 6, 3], page=1, seed=7).run().check()
    Case(8, 4, 128, lens=[700], trees=[40], page=1, seed=8, spare=5).run().check(heads=[0, 31])


@pytest.mark.parametrize("scale", [0.5, -0.3, 3.0, 1e-6])
def test_scales(scale):
    Case(8, 4, 128, lens=[300, 20], trees=[12, 20], seed=9).run(scale).check(scale, heads=[0, 9])


@pytest.mark.parametrize("spread", [30.0, 3000.0, 3e8])
def test_large_scores(spread):
    """One token takes a row, in any part; far scores too."""
    c = Case(8, 4, 128, lens=[1500, 33], trees=[10, 33], seed=10, spread=spread)
    c.run()
    scale = 1 / math.sqrt(128)
    q, out, lse = (x.double().cpu().numpy() for x in (c.q, c.out, c.lse))
    for b, (n, t) in enumerate(zip(c.lens, c.trees)):
        k, v = c.k[b].double().cpu().numpy(), c.v[b].double().cpu().numpy()
        for i in range(t):
            r = int(c.cu[b]) + i
            seen = D.tree_seen(n, t, i, c.bits[r])
            for h in (0, 17):
                kk, vv = k[:, h // 4], v[:, h // 4]
                want, wl, w = D.tree_attend(q[r, h], kk, vv, seen, scale)
                el = scale * float(np.max(np.abs(kk[seen]) @ np.abs(q[r, h]))) * 144 * 2.0 ** -24
                assert abs(lse[r, h] - wl) <= el + n * 2.0 ** -23 + 9 * 2.0 ** -20 + abs(wl) * 2.0 ** -22
                # scores are off by el: only what cannot tip is compared
                gap = np.sort(scale * (kk[seen] @ q[r, h]))
                if len(gap) < 2 or gap[-1] - gap[-2] > 2 * el + 60:
                    assert np.all(np.abs(out[r, h] - want) <= np.abs(want) * 2.0 ** -7 + 1e-12)
    assert c.ctx.status() == 0


def test_hidden_places_hold_what_they_hold():
    """NaN and infinities in K and V of drafts: rows that do not see them have the same bits as without, those that do
    see a NaN or infinity in the same elements. (Slots that no token has filled are NaN in every test here.)"""
    for G, HKV, lens, trees in ((4, 8, [300, 60], [20, 60]), (2, 4, [1700], [90])):
        d = 128 if G == 4 else 64
        plain, odd = Case(HKV, G, d, lens, trees, seed=11), Case(HKV, G, d, lens, trees, seed=11)
        plain.run().check(heads=[0])
        spoilt = {}
        for b, (j, what) in enumerate([(7, float("nan")), (11, float("inf"))][:len(lens)]):
            pos = lens[b] - trees[b] + j
            page, slot = int(odd.table[b, pos // 16]), pos % 16
            odd.v_pool[page, 1, slot, 5] = what
            odd.v_pool[page, 1, slot, d - 1] = -what
            odd.k_pool[page, 0, slot, 3] = float("nan")
            spoilt[b] = j
        odd.run()
        for b, j in spoilt.items():
            for i in range(trees[b]):
                r = int(odd.cu[b]) + i
                sees = odd.bits[r] >> j & 1
                a, o = plain.out[r], odd.out[r]
                if not sees:
                    assert torch.equal(a, o) and torch.equal(plain.lse[r], odd.lse[r]), (b, i)
                    continue
                assert bool(torch.isnan(o[:G]).all()) and bool(torch.isnan(odd.lse[r, :G]).all())   # scores of KV head 0
                bad = ~torch.isfinite(o[G:2 * G])
                want = torch.zeros_like(bad)
                want[:, 5] = want[:, d - 1] = True
                assert torch.equal(bad, want) and torch.equal(a[2 * G:], o[2 * G:]), (b, i)
                assert torch.equal(plain.lse[r, G:], odd.lse[r, G:])
        assert odd.ctx.status() == 0


def test_prefix_values_that_are_not_finite():
    c = Case(8, 4, 128, lens=[400], trees=[10], seed=12)
    page, slot = int(c.table[0, 3]), 5
    c.v_pool[page, 2, slot, 9] = float("inf")
    c.run()
    bad = ~torch.isfinite(c.out)
    want = torch.zeros_like(bad)
    want[:, 8:12, 9] = True
    assert torch.equal(bad, want)


def test_rows_do_not_depend_on_their_neighbours():
    """The same tree alone and among others, and its first rows without its last, give the same bits where the shares
    of the key tiles fall alike (one key tile to a block)."""
    lens, trees = [100, 90, 80], [30, 17, 64]
    c = Case(8, 4, 128, lens=lens, trees=trees, seed=13)
    c.run()
    first = c.out.clone()
    c.out.fill_(7.0)
    c.q[int(c.cu[1]):int(c.cu[2])] = float("nan")
    c.run()
    keep = [r for r in range(int(c.cu[-1])) if not c.cu[1] <= r < c.cu[2]]
    assert torch.equal(first[keep], c.out[keep])


def test_same_bits_every_time():
    c = Case(4, 7, 128, lens=[9000, 3001], trees=[30, 70], seed=14)
    c.run()
    a, b = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(0)
        c.run()
        assert torch.equal(a, c.out) and torch.equal(b, c.lse)


def test_errors_are_recorded():
    T = tsl()
    SEQ, OOB = T.STATUS_CODE["TS_ERR_SEQ_LEN"], T.STATUS_CODE["TS_ERR_PAGE_OOB"]

    def fresh():
        return Case(8, 4, 128, lens=[200, 150, 40], trees=[8, 6, 5], seed=15)

    good = fresh().run()
    # a length below the drafts, above the maximum, negative: that sequence alone is left as it is
    for bad in (3, 10 ** 6, -1):
        c = fresh().run(lens=[200, bad, 40])
        assert c.ctx.status() == SEQ
        assert torch.all(c.out[8:14] == 7.0) and torch.all(c.lse[8:14] == 7.0)
        for rows in (slice(0, 8), slice(14, 19)):
            assert torch.allclose(c.out[rows].float(), good.out[rows].float(), atol=0.02)
    # boundaries that descend or end beyond the rows
    c = fresh().run(cu=[0, 8, 4, 19])
    assert c.ctx.status() == SEQ and torch.allclose(c.out[:4].float(), good.out[:4].float(), atol=0.02)
    c = fresh().run(cu=[0, 8, 14, 1000])
    assert c.ctx.status() == SEQ and torch.all(c.out[14:] == 7.0)
    c = fresh().run(cu=[2, 8, 14, 19])
    assert c.ctx.status() == SEQ and torch.all(c.out[:8] == 7.0)
    # pages outside the pool: their tokens are left out (one among the prefix, one that holds drafts)
    c = fresh()
    table = c.table.copy()
    table[0, 2], table[1, 9] = c.pages, -1
    c.run(table=table)
    assert c.ctx.status() == OOB
    c.check(hidden={0: list(range(32, 48)), 1: list(range(144, 150))}, heads=[0, 31])
    # every page of a sequence outside the pool
    c = fresh()
    table = c.table.copy()
    table[2] = 10 ** 6
    c.run(table=table)
    assert c.ctx.status() == OOB and torch.all(c.out[14:19] == 0) and torch.all(c.lse[14:19] == -math.inf)
    # more drafts than the mask has words for
    c = Case(8, 4, 128, lens=[200, 150], trees=[40, 3], seed=16)
    c.words = 1
    c.run()
    assert c.ctx.status() == SEQ and torch.all(c.out[:40] == 7.0) and not torch.any(c.out[40:] == 7.0).item()


def test_captured_and_replayed_and_on_another_stream():
    c = Case(8, 4, 128, lens=[3000, 200], trees=[20, 33], seed=17)
    c.run()
    want, wl = c.out.clone(), c.lse.clone()
    table, lens, cu, mask = c.dev(c.table), c.dev(c.lens), c.dev(c.cu), c.mask_tensor()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(0)
    torch.cuda.synchronize()
    c.ctx.tree_attend(c.q, c.k_pool, c.v_pool, table, lens, cu, mask, c.out, c.lse, stream=s)
    s.synchronize()
    assert torch.equal(c.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.ctx.tree_attend(c.q, c.k_pool, c.v_pool, table, lens, cu, mask, c.out, c.lse)
    for _ in range(2):
        c.out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(c.lse, wl)
    # lengths may change between replays: they are read on the device
    lens.sub_(torch.tensor([1000, 0], dtype=torch.int32, device=DEV))
    mask.fill_(-1)
    g.replay()
    torch.cuda.synchronize()
    c.k[0], c.v[0], c.lens = c.k[0][:2000], c.v[0][:2000], [2000, 200]
    c.bits = [(1 << t) - 1 for t in c.trees for _ in range(t)]
    c.check(heads=[0, 31])


def test_strided_outputs_and_unsupported_contexts():
    T = tsl()
    c = Case(4, 2, 64, lens=[100], trees=[10], seed=18)
    wide = torch.full((10, 8 * 64 + 16), 7.0, dtype=BF, device=DEV)
    c.out = wide[:, :512].view(10, 8, 64)
    c.run().check()
    assert torch.all(wide[:, 512:] == 7.0)
    q4 = T.Context(8, 4, 64, T.TS_KV_Q4, 1, 8, 8)
    pool = torch.zeros(8, 4, 16 * 34, dtype=torch.uint8, device=DEV)
    with pytest.raises(T.TokenSelectError) as e:
        q4.tree_attend(c.q, pool, pool, torch.zeros(1, 8, dtype=torch.int32, device=DEV), c.dev([100]), c.dev([0, 10]), None, c.out)
    assert e.value.status == T.STATUS_CODE["TS_ERR_UNSUPPORTED"]
