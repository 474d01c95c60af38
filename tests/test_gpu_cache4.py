"""The 4-bit paged cache on the GPU: rows in and out (exact), the score, the attention over the whole
cache and over a selection, and a whole decode step, against the fp64 oracle.

Tolerances (u24 = 2^-24 and so on). A logit is a sum of d products that are exact in fp32, of a query
held in two fp16 terms (2^-22 of the head's largest element) and scaled: off by at most
el = alpha sum|q_e k_e| (d + 16) u24 + alpha max|q| sum|k_e| 2^-21. A weight is off by twice that and
2^-20 for its exponential, relatively; times its scale it enters the output as two fp16 terms (2^-21, or
2^-31 of the largest such product, 7 of which a code may be). Sums of n terms in fp32 add at most n 2^-23
of the sum of magnitudes.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GEOS = [(4, 4, 64), (32, 8, 128), (28, 4, 128), (9, 1, 64), (32, 2, 128), (3, 3, 128), (10, 5, 64), (80, 40, 64)]


class Cache:
    """A 4-bit cache of random rows, written through the library; pages scattered, tails never written."""

    def __init__(self, H, Hkv, d, lens, seed=0, spread=1.0, poison=True):
        self.T = T = tsl()
        rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.d, self.lens, self.B = H, Hkv, d, lens, len(lens)
        np_ = [(n + 15) // 16 for n in lens]
        self.pages = sum(np_) + 3
        perm = rng.permutation(self.pages)
        self.table = np.full((self.B, max(1, max(np_)) + 1), -7, dtype=np.int32)
        at = 0
        for b, x in enumerate(np_):
            self.table[b, :x] = perm[at:at + x]
            at += x
        self.pt = torch.from_numpy(self.table).to(DEV)
        self.ctx = T.Context(H, Hkv, d, T.TS_KV_Q4, self.B, self.table.shape[1], self.pages)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rows = sum(lens)
        self.k = (torch.randn(rows, Hkv, d, generator=g, device=DEV) * spread).to(torch.bfloat16)
        self.v = torch.randn(rows, Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
        self.q = torch.randn(self.B, H, d, generator=g, device=DEV)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        self.seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
        # slots that no row was written to hold NaN scales
        fill = 255 if poison else 0
        blk = 16 * (d // 2 + d // 32)
        self.kp, self.vp = (torch.full((self.pages, Hkv, blk), fill, dtype=torch.uint8, device=DEV) for _ in range(2))
        if rows:
            self.ctx.append_prompt(self.k, self.v, self.cu, self.pt, self.kp, self.vp)
        assert self.ctx.status() == 0
        self.kval = O.q4_pool_values(self.kp.cpu().numpy(), d)
        self.vval = O.q4_pool_values(self.vp.cpu().numpy(), d)

    def rows(self, val, b, g, tokens):
        t = np.asarray(tokens)
        return val[self.table[b, t // 16], g, t % 16]

    def check(self, out, lse, b, tokens, scale=None):
        scale = scale or 1 / math.sqrt(self.d)
        n = len(tokens)
        for h in range(self.H):
            g = h // (self.H // self.Hkv)
            if n == 0:
                assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf
                continue
            q = self.q[b, h].double().cpu().numpy()
            k, v = self.rows(self.kval, b, g, tokens), self.rows(self.vval, b, g, tokens)
            want, wl, w = O.attention(q, k, v, scale)
            el = abs(scale) * float(np.max(np.abs(k) @ np.abs(q) * (self.d + 16) * 2.0 ** -24
                                           + np.abs(k).sum(1) * np.abs(q).max() * 2.0 ** -21))
            big = 7 * n * float(np.max(w[:, None] * np.abs(v))) * 2.0 ** -31
            tol = (w @ np.abs(v)) * (2 * el + 2.0 ** -21 + 2.0 ** -20 + n * 2.0 ** -23) + big + 1e-30
            assert np.all(np.abs(out[b, h] - want) <= tol), (b, h, np.max(np.abs(out[b, h] - want) / tol))
            assert abs(lse[b, h] - wl) <= el + n * 2.0 ** -23 + 2.0 ** -20 + abs(wl) * 2.0 ** -22


@pytest.mark.parametrize("H,Hkv,d", GEOS)
def test_rows_written_are_the_oracle_s_bytes_and_read_back_as_their_values(H, Hkv, d):
    lens = [1, 33, 0, 16, 70]
    c = Cache(H, Hkv, d, lens, seed=H + d, poison=False)
    cu = np.concatenate([[0], np.cumsum(lens)])
    for x, pool in ((c.k, c.kp), (c.v, c.vp)):
        codes, scale = O.q4_quantise(x.double().cpu().numpy())
        want = np.zeros(pool.shape, dtype=np.uint8)
        for b, n in enumerate(lens):
            for p in range((n + 15) // 16):
                m = min(16, n - 16 * p)
                for g in range(Hkv):
                    full = np.zeros((16, d // 64, 64), dtype=np.int64)
                    sc = np.zeros((16, d // 64))
                    full[:m], sc[:m] = (y[cu[b] + 16 * p:cu[b] + 16 * p + m, g] for y in (codes, scale))
                    want[c.table[b, p], g] = O.q4_pack(full, sc)
        assert np.array_equal(pool.cpu().numpy(), want)
    ko, vo = (torch.full((sum(lens), Hkv, d), 5.0, device=DEV) for _ in range(2))
    c.ctx.read_kv(c.cu, c.pt, c.kp, c.vp, ko, vo)
    assert c.ctx.status() == 0
    for x, o in ((c.k, ko), (c.v, vo)):
        assert np.array_equal(o.double().cpu().numpy(), O.q4_values(*O.q4_quantise(x.double().cpu().numpy())))


def test_quantised_special_groups():
    c = Cache(2, 1, 128, [8], seed=1)
    k = torch.zeros(8, 1, 128, dtype=torch.bfloat16, device=DEV)
    k[1, 0, 3] = float("nan")
    k[2, 0, 70] = float("inf")
    k[3, 0, 0] = 1e-39                                # a subnormal: scale rounded in bf16's subnormals
    k[4, 0, :4] = torch.tensor([7.0, 0.5, 1.5, -2.5])
    k[5, 0, 64] = 3.38e38
    k[6, 0, 9] = -0.0
    c.ctx.append_prompt(k, k, c.cu, c.pt, c.kp, c.vp)
    ko, vo = (torch.zeros(8, 1, 128, device=DEV) for _ in range(2))
    c.ctx.read_kv(c.cu, c.pt, c.kp, c.vp, ko, vo)
    want = O.q4_values(*O.q4_quantise(k.double().cpu().numpy()))
    assert np.array_equal(ko.double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[1, 0, :64]).all() and (want[1, 0, 64:] == 0).all() and np.isnan(want[2, 0, 64:]).all()


def test_append_single_tokens_and_prompts_behind_one_another():
    # a prompt, then tokens one by one, then a second prompt: the same bytes as all rows at once
    T = tsl()
    H, Hkv, d, total = 8, 2, 128, 61
    c = Cache(H, Hkv, d, [total], seed=3, poison=False)
    kp, vp = torch.zeros_like(c.kp), torch.zeros_like(c.vp)
    one = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    c.ctx.append_prompt(c.k[:20], c.v[:20], one, c.pt, kp, vp)
    for t in range(20, 27):
        c.ctx.append_kv(c.k[t:t + 1], c.v[t:t + 1], c.pt, torch.tensor([t + 1], dtype=torch.int32, device=DEV), kp, vp)
    rest = torch.tensor([0, total - 27], dtype=torch.int32, device=DEV)
    c.ctx.append_prompt(c.k[27:], c.v[27:], rest, c.pt, kp, vp, starts=torch.tensor([27], dtype=torch.int32, device=DEV))
    assert c.ctx.status() == 0
    assert torch.equal(kp, c.kp) and torch.equal(vp, c.vp)
    # strided rows: k and v as column ranges of one matrix
    wide = torch.randn(total, (H + 2 * Hkv) * d, device=DEV).to(torch.bfloat16)
    kk, vv = wide[:, H * d:(H + Hkv) * d].view(total, Hkv, d), wide[:, (H + Hkv) * d:].view(total, Hkv, d)
    kp2, vp2, kp3, vp3 = (torch.zeros_like(c.kp) for _ in range(4))
    c.ctx.append_prompt(kk, vv, c.cu, c.pt, kp2, vp2)
    c.ctx.append_prompt(kk.contiguous(), vv.contiguous(), c.cu, c.pt, kp3, vp3)
    assert torch.equal(kp2, kp3) and torch.equal(vp2, vp3)
    assert T.ts_page_bytes(c.ctx.cfg) == c.kp[0].numel()


@pytest.mark.parametrize("kind,page_size", [("f32", 16), ("bf16", 16), ("bf16", 1), ("f32", 1)])
def test_append_prompt_and_read_into_the_other_pools(kind, page_size):
    T = tsl()
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    H, Hkv, d, lens, starts = 4, 2, 64, [5, 0, 40], [3, 7, 16]
    H, Hkv = (8, 2) if kind == "f32" else (8, 4)
    mp = 64 // page_size
    ctx = T.Context(H, Hkv, d, T.TS_KV_F32 if kind == "f32" else T.TS_KV_BF16, 3, mp, 3 * mp, page_size=page_size)
    table = torch.randperm(3 * mp).view(3, mp).to(torch.int32).to(DEV)
    k, v = (torch.randn(50, Hkv, d, device=DEV).to(dt) for _ in range(2))       # five rows behind the last sequence
    cu = torch.tensor([0, 5, 5, 45], dtype=torch.int32, device=DEV)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    kp, vp = (torch.full((3 * mp, Hkv, page_size, d), 9.0, device=DEV).to(dt) for _ in range(2))
    want_k, want_v = kp.clone(), vp.clone()
    ctx.append_prompt(k, v, cu, table, kp, vp, starts=st)
    for b, (lo, hi) in enumerate([(0, 5), (5, 5), (5, 45)]):
        for r in range(lo, hi):
            pos = starts[b] + r - lo
            want_k[table[b, pos // page_size], :, pos % page_size] = k[r]
            want_v[table[b, pos // page_size], :, pos % page_size] = v[r]
    assert ctx.status() == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    ko, vo = (torch.full((50, Hkv, d), -3.0, device=DEV) for _ in range(2))
    ctx.read_kv(cu, table, kp, vp, ko, vo, starts=st)
    assert torch.equal(ko[:45], k[:45].float()) and torch.equal(vo[:45], v[:45].float())
    assert (ko[45:] == -3).all() and (vo[45:] == -3).all()


def test_rows_without_a_place_are_reported_and_left_out():
    T = tsl()
    c = Cache(4, 2, 64, [30, 20], seed=9, poison=False)
    SEQ, PAGE = T.STATUS_CODE["TS_ERR_SEQ_LEN"], T.STATUS_CODE["TS_ERR_PAGE_OOB"]

    def append(cu, starts=None, table=None):
        kp, vp = torch.zeros_like(c.kp), torch.zeros_like(c.vp)
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
        c.ctx.append_prompt(c.k, c.v, cu, c.pt if table is None else table, kp, vp, starts=st)
        return c.ctx.status(), kp, vp

    st, kp, vp = append([0, 30, 50])
    assert st == 0 and torch.equal(kp, c.kp)
    st, kp, _ = append([0, 30, 51])                            # ends beyond the rows: none of its rows
    assert st == SEQ
    first = torch.zeros_like(kp)
    for p in range(2):
        first[c.table[0, p]] = c.kp[c.table[0, p]]
    assert torch.equal(kp, first)
    assert append([0, 30, 20])[0] == SEQ                       # descends
    assert append([3, 30, 50])[0] == SEQ                       # does not begin at 0
    st, kp, _ = append([0, 30, 50], starts=[c.ctx.max_tokens - 10, -1])
    assert st == SEQ                                           # past the last position, before the first
    bad = c.pt.clone()
    bad[0, 1] = c.pages
    bad[1, 0] = -1
    st, kp, _ = append([0, 30, 50], table=bad)
    assert st == PAGE
    keep = torch.zeros_like(c.kp)
    for b, p in ((0, 0), (1, 1)):
        keep[c.table[b, p]] = c.kp[c.table[b, p]]
    assert torch.equal(kp, keep)
    one = torch.zeros_like(c.kp)
    c.ctx.append_kv(c.k[:2], c.v[:2], c.pt, torch.tensor([0, 10 ** 6], dtype=torch.int32, device=DEV), one, one.clone())
    assert c.ctx.status() == SEQ and not one.any()


@pytest.mark.parametrize("H,Hkv,d", GEOS)
@pytest.mark.parametrize("lens", [[1], [0, 16, 17, 15], [300, 1, 0, 2049, 31]])
def test_attend_over_the_whole_cache(H, Hkv, d, lens):
    c = Cache(H, Hkv, d, lens, seed=H * 7 + sum(lens), spread=2.0)
    out, lse = torch.full((c.B, H, d), 7.0, device=DEV), torch.full((c.B, H), 7.0, device=DEV)
    c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse)
    assert c.ctx.status() == 0
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        c.check(o, z, b, np.arange(n))
    # the same bits again, without lse, and through a captured graph on another stream
    out2 = torch.zeros_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out2)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out2)
        out2.zero_()
        g.replay()
    s.synchronize()
    assert torch.equal(out, out2)


def test_attend_where_the_maximum_moves_late_and_far():
    # keys grow along the sequence: every page raises the running maximum, by far more than 2^8 at the end
    c = Cache(16, 2, 128, [1500], seed=4)
    grow = torch.linspace(0.01, 30.0, 1500, device=DEV).view(-1, 1, 1)
    k = (c.q[0].view(2, 8, 128)[:, :1].squeeze(1)[None] * grow).to(torch.bfloat16)
    c.ctx.append_prompt(k, c.v, c.cu, c.pt, c.kp, c.vp)
    c.kval = O.q4_pool_values(c.kp.cpu().numpy(), 128)
    for scale in (0.0, -0.5, 0.25):
        out, lse = torch.zeros(1, 16, 128, device=DEV), torch.zeros(1, 16, device=DEV)
        c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse, scale=scale)
        c.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), 0, np.arange(1500), scale or None)


@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 64), (28, 4, 128)])
def test_attend_over_values_of_very_different_sizes(H, Hkv, d):
    # scales from 1e-12 to 1e12 along the sequence, both ways, and single rows far above the others
    n = 700
    c = Cache(H, Hkv, d, [n, n, n], seed=14)
    size = torch.logspace(-12, 12, n, device=DEV)
    outlier = torch.full((n,), 1e-3, device=DEV)
    outlier[5], outlier[333], outlier[690] = 1e6, 3e9, 0.0
    v = c.v.float().view(3, n, Hkv, d) * torch.stack([size, size.flip(0), outlier]).view(3, n, 1, 1)
    c.ctx.append_prompt(c.k, v.view(3 * n, Hkv, d).to(torch.bfloat16), c.cu, c.pt, c.kp, c.vp)
    c.vval = O.q4_pool_values(c.vp.cpu().numpy(), d)
    out, lse = torch.zeros(3, H, d, device=DEV), torch.zeros(3, H, device=DEV)
    idx = torch.arange(n, dtype=torch.int32, device=DEV).repeat(3, 1)
    for call in (lambda: c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse),
                 lambda: c.ctx.sparse_attend(c.q, c.kp, c.vp, c.pt, idx, c.seq, out, lse)):
        out.zero_()
        call()
        for b in range(3):
            c.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), b, np.arange(n))


@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (28, 4, 128)])
def test_more_sequences_than_a_kernel_keeps_at_hand(H, Hkv, d):
    # 600 sequences, most of them empty or short
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.choice([0, 0, 0, 1, 5, 16, 17, 40], 600)]
    lens[599] = 33
    c = Cache(H, Hkv, d, lens, seed=15)
    out, lse = torch.zeros(600, H, d, device=DEV), torch.zeros(600, H, device=DEV)
    c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse)
    vote = torch.zeros(600, c.ctx.max_tokens, device=DEV)
    c.ctx.score(c.q, c.kp, c.pt, c.seq, vote)
    assert c.ctx.status() == 0
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in list(range(0, 600, 37)) + [511, 512, 513, 599]:
        c.check(o, z, b, np.arange(lens[b]))
    mass = vote.double().sum(1).cpu().numpy()
    assert np.allclose(mass, [H if n else 0 for n in lens], atol=1e-4)


@pytest.mark.parametrize("H,Hkv,d", GEOS)
def test_attend_over_a_selection(H, Hkv, d):
    lens = [900, 40, 5, 0]
    c = Cache(H, Hkv, d, lens, seed=H + 1)
    rng = np.random.default_rng(2)
    sel = [np.sort(rng.permutation(900)[:333]), np.arange(40), np.array([4, 0, 4, 2]), np.array([], dtype=int)]
    idx = torch.full((4, 400), 10 ** 8, dtype=torch.int32, device=DEV)
    for b, x in enumerate(sel):
        idx[b, :len(x)] = torch.from_numpy(x).to(torch.int32).to(DEV)
    cnt = torch.tensor([len(x) for x in sel], dtype=torch.int32, device=DEV)
    out, lse = torch.zeros(4, H, d, device=DEV), torch.zeros(4, H, device=DEV)
    c.ctx.sparse_attend(c.q, c.kp, c.vp, c.pt, idx, cnt, out, lse)
    assert c.ctx.status() == 0
    for b, x in enumerate(sel):                       # (an index listed twice counts twice)
        c.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), b, x)


def test_every_token_selected_is_the_whole_cache():
    c = Cache(28, 4, 128, [777, 64], seed=8)
    idx = torch.arange(777, dtype=torch.int32, device=DEV).repeat(2, 1)
    outs = [torch.zeros(2, 28, 128, device=DEV) for _ in range(2)]
    c.ctx.sparse_attend(c.q, c.kp, c.vp, c.pt, idx, c.seq, outs[0])
    c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, outs[1])
    assert torch.allclose(outs[0], outs[1], rtol=0, atol=2.0 ** -13)


def test_attend_reports_bad_lengths_and_pages_and_leaves_them_out():
    T = tsl()
    c = Cache(8, 4, 64, [100, 50, 20], seed=6)
    seq = torch.tensor([100, -1, c.ctx.max_tokens + 1], dtype=torch.int32, device=DEV)
    out, lse = torch.ones(3, 8, 64, device=DEV), torch.ones(3, 8, device=DEV)
    c.ctx.attend(c.q, c.kp, c.vp, c.pt, seq, out, lse)
    assert c.ctx.status() == T.STATUS_CODE["TS_ERR_SEQ_LEN"]
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate([100, 0, 0]):
        c.check(o, z, b, np.arange(n))
    bad = c.pt.clone()
    bad[0, 2], bad[2, 0] = c.pages, -1
    c.ctx.attend(c.q, c.kp, c.vp, bad, c.seq, out, lse)
    assert c.ctx.status() == T.STATUS_CODE["TS_ERR_PAGE_OOB"]
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    left = [np.concatenate([np.arange(32), np.arange(48, 100)]), np.arange(50), np.arange(16, 20)]
    for b, x in enumerate(left):
        c.check(o, z, b, x)
    # through an index list too
    idx = torch.arange(100, dtype=torch.int32, device=DEV).repeat(3, 1)
    c.ctx.sparse_attend(c.q, c.kp, c.vp, bad, idx, c.seq, out, lse)
    assert c.ctx.status() == T.STATUS_CODE["TS_ERR_PAGE_OOB"]
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, x in enumerate(left):
        c.check(o, z, b, x)
    # the context stays usable
    c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse)
    assert c.ctx.status() == 0
    c.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), 0, np.arange(100))


def test_a_nan_stays_in_its_own_head_and_sequence():
    c = Cache(8, 2, 64, [70, 33], seed=12)
    k = c.k.clone()
    k[5, 1, 3] = float("nan")                          # sequence 0, KV head 1
    c.ctx.append_prompt(k, c.v, c.cu, c.pt, c.kp, c.vp)
    out, lse = torch.zeros(2, 8, 64, device=DEV), torch.zeros(2, 8, device=DEV)
    vote = torch.zeros(2, c.ctx.max_tokens, device=DEV)
    idx = torch.arange(70, dtype=torch.int32, device=DEV).repeat(2, 1)
    for call in (lambda: c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse),
                 lambda: c.ctx.sparse_attend(c.q, c.kp, c.vp, c.pt, idx, c.seq, out, lse)):
        out.zero_()
        call()
        assert torch.isnan(out[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
        assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()
    c.ctx.score(c.q, c.kp, c.pt, c.seq, vote)
    assert torch.isnan(vote[0, :70]).all() and torch.isfinite(vote[1, :33]).all()
    assert c.ctx.status() == 0


@pytest.mark.parametrize("H,Hkv,d", GEOS)
@pytest.mark.parametrize("lens", [[1], [700, 0, 16, 33], [5000]])
def test_score_against_the_oracle(H, Hkv, d, lens):
    c = Cache(H, Hkv, d, lens, seed=H + sum(lens), spread=1.5)
    q = c.q.double().cpu().numpy()
    want, tol = [], []
    for b, n in enumerate(lens):
        w, el = np.zeros(n), 0.0
        for h in range(H if n else 0):
            k = c.rows(c.kval, b, h // (H // Hkv), np.arange(n))
            w += O.attention(q[b, h], k, k, 1 / math.sqrt(d))[2]
            el = max(el, float(np.max(np.abs(k) @ np.abs(q[b, h]) * (d + 16) * 2.0 ** -24
                                      + np.abs(k).sum(1) * np.abs(q[b, h]).max() * 2.0 ** -21)) / math.sqrt(d))
        want.append(w)
        tol.append(w * (2 * el + n * 2.0 ** -23 + 2.0 ** -19))
    # all sequences, the same again (the same bits), and with the first one skipped: that row is left as
    # it is, and the others' pages are then shared out over the CTAs in another way, so their sums may
    # differ in the last bits
    votes = []
    for skipped in ([], [], [0]):
        vote = torch.full((c.B, c.ctx.max_tokens + 4), 3.0, device=DEV)
        skip = torch.tensor([int(b in skipped) for b in range(c.B)], dtype=torch.uint8, device=DEV)
        c.ctx.score(c.q, c.kp, c.pt, c.seq, vote, skip=skip if skipped else None)
        assert c.ctx.status() == 0
        votes.append(vote)
        got = vote.double().cpu().numpy()
        for b, n in enumerate(lens):
            n = 0 if b in skipped else n
            assert np.all(np.abs(got[b, :n] - want[b][:n]) <= tol[b][:n])
            assert np.all(got[b, n:] == 3.0)
    assert torch.equal(votes[0], votes[1])


@pytest.mark.parametrize("fn", ["TS_SCORE_LOGIT_SUM", "TS_SCORE_HEAD_HARD_VOTE"])
def test_the_other_selection_functions_read_the_same_logits(fn):
    T = tsl()
    c = Cache(8, 2, 128, [900], seed=5)
    vote = torch.zeros(1, c.ctx.max_tokens, device=DEV)
    c.ctx.score_fn(T.params(k=100, n_sink=4, n_local=16, score_fn=getattr(T, fn)), c.q, c.kp, c.pt, c.seq, vote)
    logits = O.head_logits(c.q[0].double().cpu().numpy(), c.kval, c.table[0], 900)
    got = vote[0, :900].double().cpu().numpy()
    if fn == "TS_SCORE_LOGIT_SUM":
        assert np.max(np.abs(got - O.logit_sum_scores(logits))) <= 1e-4
    else:
        assert np.array_equal(got, O.hard_vote_counts(logits, 900, 100, 4, 16))


def test_the_operators_together_prompt_to_decode():
    # prompts are attended and written, then decode steps append, select and attend, all over one 4-bit cache
    T = tsl()
    H, Hkv, d, lens, steps = 28, 4, 128, [600, 37], 4
    c = Cache(H, Hkv, d, [n + steps for n in lens], seed=21, poison=False)
    ctx, B = c.ctx, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    qkv = torch.randn(sum(lens), (H + 2 * Hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
    q = qkv[:, :H * d].view(-1, H, d)
    k, v = (qkv[:, (H + i * Hkv) * d:(H + (i + 1) * Hkv) * d].view(-1, Hkv, d) for i in range(2))
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=DEV)
    out = torch.zeros(sum(lens), H, d, dtype=torch.bfloat16, device=DEV)
    c.kp.zero_()
    c.vp.zero_()
    ctx.prompt_attend(q, k, v, cu, out)
    ctx.append_prompt(k, v, cu, c.pt, c.kp, c.vp)
    cache = ctx.cache(1, 64)
    prm = T.params(k=64, n_sink=4, n_local=16, theta=0.9)
    idx, cnt = torch.zeros(B, 84, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    o, full = torch.zeros(B, H, d, device=DEV), torch.zeros(B, H, d, device=DEV)
    hit = torch.zeros(B, dtype=torch.uint8, device=DEV)
    states = [O.CacheState() for _ in range(B)]
    qt = torch.randn(B, H, d, generator=g, device=DEV)
    hits = 0
    for t in range(steps):
        seq = torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device=DEV)
        kn, vn = (torch.randn(B, Hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        if t != 2:
            qt = qt + 0.1 * torch.randn(B, H, d, generator=g, device=DEV)
        else:
            qt = torch.randn(B, H, d, generator=g, device=DEV)
        ctx.append_kv(kn, vn, c.pt, seq, c.kp, c.vp)
        ctx.decode_step(qt, c.kp, c.vp, c.pt, seq, prm, idx, cnt, o, hit=hit, cache=cache)
        ctx.attend(qt, c.kp, c.vp, c.pt, seq, full)
        assert ctx.status() == 0
        kv, vv = O.q4_pool_values(c.kp.cpu().numpy(), d), O.q4_pool_values(c.vp.cpu().numpy(), d)
        for b in range(B):
            n = lens[b] + t + 1
            ref = O.decode_step(states[b], qt[b].double().cpu().numpy(), kv, vv, c.table[b], n, k=64, n_sink=4,
                                n_local=16, theta=0.9)
            assert bool(hit[b]) == ref["hit"]
            hits += ref["hit"]
            assert np.array_equal(idx[b, :int(cnt[b])].cpu().numpy(), ref["idx"])
            got = o[b].double().cpu().numpy()
            assert np.max(np.abs(got - ref["out"])) <= 2e-3 * np.max(np.abs(ref["out"]))
            dense = O.dense_attention(qt[b].double().cpu().numpy(), kv, vv, c.table[b], n)
            dense = dense[0] if isinstance(dense, tuple) else dense
            assert np.max(np.abs(full[b].double().cpu().numpy() - dense)) <= 2e-3 * np.max(np.abs(dense))
    assert 0 < hits < 2 * steps
    assert torch.isfinite(out).all()


def _far_calls(ctx, T, k, v, kn, vn, q, cu, table, kp, vp, n):
    """Everything that reads or writes pages, over the pages of `table`; what it gives."""
    H, d = q.shape[1:]
    Hkv = k.shape[1]
    q4 = ctx.cfg.kv_dtype == T.TS_KV_Q4
    seq = torch.tensor([n + 1], dtype=torch.int32, device=DEV)
    ctx.append_prompt(k, v, cu, table, kp, vp)
    ctx.append_kv(kn, vn, table, seq, kp, vp)
    ko, vo = torch.zeros(n + 1, Hkv, d, device=DEV), torch.zeros(n + 1, Hkv, d, device=DEV)
    ctx.read_kv(torch.tensor([0, n + 1], dtype=torch.int32, device=DEV), table, kp, vp, ko, vo)
    got = [ko, vo]
    if q4:
        vote = torch.zeros(1, ctx.max_tokens, device=DEV)
        ctx.score(q, kp, table, seq, vote)
        idx = torch.arange(0, n + 1, 3, dtype=torch.int32, device=DEV).view(1, -1)
        cnt = torch.tensor([idx.shape[1]], dtype=torch.int32, device=DEV)
        o = [torch.zeros(1, H, d, device=DEV) for _ in range(2)]
        ctx.attend(q, kp, vp, table, seq, o[0])
        ctx.sparse_attend(q, kp, vp, table, idx, cnt, o[1])
        got += [vote[:, :n + 1], *o]
    assert ctx.status() == 0
    return [x.clone() for x in got]


@pytest.mark.parametrize("kind,pages", [("TS_KV_Q4", 520_000), ("TS_KV_F32", 70_000)])
def test_pages_past_four_gigabytes(kind, pages):
    T = tsl()
    H, Hkv, d, n = 32, 8, 128, 90
    kv_dtype = getattr(T, kind)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    rows = [torch.randn(m, Hkv, d, generator=g, device=DEV) for m in (n, n, 1, 1)]
    if kv_dtype == T.TS_KV_Q4:
        rows = [x.to(torch.bfloat16) for x in rows]
    q = torch.randn(1, H, d, generator=g, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    results = []
    for num, first in ((pages, pages - 6), (6, 0)):
        ctx = T.Context(H, Hkv, d, kv_dtype, 1, 6, num)
        size = num * T.ts_page_bytes(ctx.cfg)
        assert num == 6 or size > 1 << 32
        kp, vp = (torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2))
        table = (first + torch.tensor([[5, 0, 3, 1, 4, 2]], device=DEV)).to(torch.int32)
        results.append(_far_calls(ctx, T, *rows, q, cu, table, kp, vp, n))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_a_decode_chain_captured_once_and_replayed_over_growing_sequences():
    # append, decode step and attention of the whole cache as one graph on a stream of its own; lengths, rows and
    # queries change between replays, and eager calls run in between over the same context
    T = tsl()
    H, Hkv, d, lens, steps = 32, 8, 128, [300, 1, 47], 20
    a, b = (Cache(H, Hkv, d, [n + steps for n in lens], seed=31, poison=False) for _ in range(2))
    B = len(lens)
    prm = T.params(k=32, n_sink=4, n_local=16, theta=0.9)

    def state(c):
        z = dict(idx=torch.zeros(B, 52, dtype=torch.int32, device=DEV), cnt=torch.zeros(B, dtype=torch.int32, device=DEV),
                 o=torch.zeros(B, H, d, device=DEV), full=torch.zeros(B, H, d, device=DEV), lse=torch.zeros(B, H, device=DEV))
        z.update(q=torch.zeros(B, H, d, device=DEV), kn=torch.zeros(B, Hkv, d, dtype=torch.bfloat16, device=DEV),
                 vn=torch.zeros(B, Hkv, d, dtype=torch.bfloat16, device=DEV), seq=torch.ones(B, dtype=torch.int32, device=DEV),
                 cache=c.ctx.cache(1, 52))
        return z

    def chain(c, z):
        c.ctx.append_kv(z["kn"], z["vn"], c.pt, z["seq"], c.kp, c.vp)
        c.ctx.decode_step(z["q"], c.kp, c.vp, c.pt, z["seq"], prm, z["idx"], z["cnt"], z["o"], cache=z["cache"])
        c.ctx.attend(z["q"], c.kp, c.vp, c.pt, z["seq"], z["full"], z["lse"])

    warm = Cache(H, Hkv, d, [20] * B, seed=1, poison=False)
    chain(warm, state(warm))
    za, zb = state(a), state(b)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            chain(a, za)
    torch.cuda.synchronize()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for t in range(steps):
        new = dict(q=torch.randn(B, H, d, generator=g, device=DEV),
                   kn=torch.randn(B, Hkv, d, generator=g, device=DEV).to(torch.bfloat16),
                   vn=torch.randn(B, Hkv, d, generator=g, device=DEV).to(torch.bfloat16),
                   seq=torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device=DEV))
        for z in (za, zb):
            for name, x in new.items():
                z[name].copy_(x)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        chain(b, zb)
        if t % 5 == 0:                                 # an eager call in between uses the same scratch
            a.ctx.attend(za["q"], a.kp, a.vp, a.pt, za["seq"], torch.empty_like(za["full"]))
        for name in ("idx", "cnt", "o", "full", "lse"):
            assert torch.equal(za[name], zb[name]), (t, name)
    assert a.ctx.status() == 0 and b.ctx.status() == 0


def test_calls_that_the_context_does_not_serve():
    T = tsl()
    c = Cache(8, 4, 64, [20], seed=2)
    bf = T.Context(8, 4, 64, T.TS_KV_BF16, 1, 4, 4)
    f32 = T.Context(8, 2, 64, T.TS_KV_F32, 1, 4, 4)
    out = torch.zeros(1, 8, 64, device=DEV)
    idx, cnt = torch.zeros(1, 8, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def refused(code, fn, *a, **kw):
        with pytest.raises(T.TokenSelectError) as e:
            fn(*a, **kw)
        assert e.value.status == T.STATUS_CODE[code]

    refused("TS_ERR_UNSUPPORTED", bf.attend, c.q, c.kp, c.vp, c.pt, c.seq, out)
    refused("TS_ERR_UNSUPPORTED", f32.attend, c.q, c.kp, c.vp, c.pt, c.seq, out)
    refused("TS_ERR_INVALID_ARG", c.ctx.attend, c.q, c.kp, c.vp, c.pt, c.seq, out, scale=float("nan"))
    refused("TS_ERR_SHAPE", T.ts_attend, c.ctx.handle, c.q, c.kp, c.vp, c.pt, c.seq, 2, 0.0, out)
    refused("TS_ERR_SHAPE", T.ts_attend, c.ctx.handle, c.q, c.kp, c.vp, c.pt, c.seq, 0, 0.0, out)
    refused("TS_ERR_INVALID_ARG", T.ts_attend, c.ctx.handle, c.q, c.kp.data_ptr() + 8, c.vp, c.pt, c.seq, 1, 0.0, out)
    refused("TS_ERR_UNSUPPORTED", c.ctx.prefill_chunk, c.q.view(1, 1, 8, 64), c.kp, c.vp, c.pt, c.seq, T.params(), idx,
            cnt, out.view(1, 1, 8, 64))
    k = c.k
    refused("TS_ERR_SHAPE", T.ts_append_prompt, c.ctx.handle, k, 128, k, 256, c.cu, None, 1, 20, c.pt, c.kp, c.vp)
    refused("TS_ERR_INVALID_ARG", T.ts_append_prompt, c.ctx.handle, k, 260, k, 256, c.cu, None, 1, 20, c.pt, c.kp, c.vp)
    refused("TS_ERR_SHAPE", T.ts_append_prompt, c.ctx.handle, k, 256, k, 256, c.cu, None, 1, -1, c.pt, c.kp, c.vp)
    refused("TS_ERR_SHAPE", T.ts_append_prompt, c.ctx.handle, k, 256, k, 256, c.cu, None, 2, 20, c.pt, c.kp, c.vp)
    refused("TS_ERR_INVALID_ARG", T.ts_read_kv, c.ctx.handle, c.cu, None, 1, 20, c.pt, c.kp, c.vp, None, out)
    rows = torch.zeros(20, 4, 64, device=DEV)
    for call in (lambda: c.ctx.append_prompt(k.float(), k, c.cu, c.pt, c.kp, c.vp),
                 lambda: c.ctx.append_prompt(k, k[:9], c.cu, c.pt, c.kp, c.vp),
                 lambda: c.ctx.append_prompt(k, k, c.cu, c.pt, c.kp, c.vp, starts=c.cu),
                 lambda: c.ctx.read_kv(c.cu, c.pt, c.kp, c.vp, rows, rows[:9]),
                 lambda: c.ctx.read_kv(c.cu, c.pt, c.kp, c.vp, rows, rows.to(torch.bfloat16))):
        with pytest.raises(T.TokenSelectError):
            call()
    T.ts_append_prompt(c.ctx.handle, k, 256, k, 256, c.cu, None, 1, 0, c.pt, c.kp, c.vp)      # no rows: nothing to do
    assert c.ctx.status() == 0
