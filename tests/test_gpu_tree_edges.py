"""ts_tree_attend on the GPU: places that hold no number in parts of their own, rows by themselves and among others, long
sequences, and waits that run out."""
import pytest
import torch

from parity import tsl
from test_gpu_tree import BF, DEV, Case

pytestmark = pytest.mark.gpu


def _place(c, b, pos):
    return int(c.table[b, pos // c.page]), pos % c.page


@pytest.mark.parametrize("n", [100, 256, 385, 513, 641, 1025, 5000, 40001])
@pytest.mark.parametrize("HKV,G,d", [(8, 4, 128), (4, 2, 64)])
def test_a_key_that_is_no_number_spoils_the_rows_that_see_it(HKV, G, d, n):
    """A NaN key that is the only seen token of its part of a block (385, 513, ...: the last key tile holds it alone), and one
    among others: the outputs and sums of the rows that see it are NaN, wherever the shares of the CTAs fall."""
    for t, spoilt in ((1, n - 1), (3, n - 1), (3, n - 2), (2, 40)):
        c = Case(HKV, G, d, lens=[n], trees=[t], mask=None, seed=n)
        page, slot = _place(c, 0, spoilt)
        c.k_pool[page, 1, slot, 7] = float("nan")
        c.run()
        sees = [n - t + i >= spoilt for i in range(t)]
        out, lse = torch.isnan(c.out).all(-1), torch.isnan(c.lse)
        want = torch.zeros_like(out)
        for i in range(t):
            want[i, G:2 * G] = sees[i]
        assert torch.equal(out, want) and torch.equal(lse, want), (t, spoilt)
        assert not bool(torch.isnan(c.out).any(-1)[~want].any()) and c.ctx.status() == 0


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [120, 250, 700, 20000])
def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it_whatever_its_weight(what, n):
    """A NaN or infinite value of a token whose weight vanishes in fp32 (its score lies 700 below the others'): not finite in
    every row that sees it, in a part of its own or not; a draft's reaches those alone whose mask has it."""
    for hidden in (False, True):
        c = Case(8, 4, 128, lens=[n], trees=[4], mask=lambda t, i, rng: 15 if i % 2 else 15 & ~4, seed=n)
        c.q.fill_(8.0)
        c.k_pool.nan_to_num_(0.0)
        c.k_pool.zero_()
        pos = n - 2 if hidden else 5
        page, slot = _place(c, 0, pos)
        first = pos // 128 * 128
        for p in range(first, min(n, first + 128)):                # the whole key tile weighs nothing beside the others
            at = _place(c, 0, p)
            if n > 128 or p == pos:
                c.k_pool[at[0], :, at[1]] = -8.0
        c.v_pool[page, 2, slot, 11] = what
        c.run()
        bad = ~torch.isfinite(c.out)
        want = torch.zeros_like(bad)
        for i in range(4):
            want[i, 8:12, 11] = not hidden or i % 2 == 1
        assert torch.equal(bad, want) and bool(torch.isfinite(c.lse).all()) and c.ctx.status() == 0


def _alone(c, b, drafts):
    """The first drafts of sequence b by themselves: outputs and sums."""
    T, r0 = tsl(), int(c.cu[b])
    ctx = T.Context(c.H, c.HKV, c.d, T.TS_KV_BF16, 1, c.table.shape[1], c.pages, c.page)
    rows = slice(r0, r0 + drafts)
    out, lse = torch.full((drafts, c.H, c.d), 7.0, dtype=BF, device=DEV), torch.full((drafts, c.H), 7.0, device=DEV)
    n = c.lens[b] - c.trees[b] + drafts
    ctx.tree_attend(c.q[rows], c.k_pool, c.v_pool, c.dev(c.table[b:b + 1]), c.dev([n]), c.dev([0, drafts]),
                    c.mask_tensor()[rows].contiguous(), out, lse)
    assert ctx.status() == 0
    return out, lse


def test_a_tree_alone_and_without_its_last_rows():
    """The same bits alone and among others, and for a tree's first drafts without its last, where every block has one key
    tile (the shares of the key tiles fall alike)."""
    c = Case(8, 4, 128, lens=[100, 90, 80, 128], trees=[30, 17, 64, 90], seed=23)
    c.run()
    for b, t in enumerate(c.trees):
        for drafts in (t, t - 1, t // 2, 1):
            out, lse = _alone(c, b, drafts)
            rows = slice(int(c.cu[b]), int(c.cu[b]) + drafts)
            assert torch.equal(out, c.out[rows]) and torch.equal(lse, c.lse[rows]), (b, drafts)


@pytest.mark.parametrize("HKV,G,d,t,page", [(8, 4, 128, 64, 16), (4, 2, 64, 20, 16), (2, 8, 128, 9, 1)])
def test_long_sequences(HKV, G, d, t, page):
    """131,057 tokens: key tiles of a KV head over a dozen CTAs and more."""
    c = Case(HKV, G, d, lens=[131057], trees=[t], page=page, seed=24)
    c.run().check(rows=[0, t // 2, t - 1], heads=[0, HKV * G - 1])


def test_waits_that_run_out_are_reported():
    """A limit that the first products cannot keep: the status says so, what follows is right."""
    T = tsl()
    c = Case(8, 4, 128, lens=[131057, 300, 64], trees=[20, 33, 5], seed=25)
    c.run()
    assert c.ctx.status() == 0
    want, wl = c.out.clone(), c.lse.clone()
    for _ in range(3):
        T.ts_set_wait_limit(c.ctx.handle, 1)
        c.run()
        assert c.ctx.status() == T.STATUS_CODE["TS_ERR_TIMEOUT"]
        T.ts_set_wait_limit(c.ctx.handle, 1000000000)
        c.out.fill_(0)
        c.run()
        assert c.ctx.status() == 0 and torch.equal(c.out, want) and torch.equal(c.lse, wl)
