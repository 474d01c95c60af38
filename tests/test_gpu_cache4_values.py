"""Values over a 4-bit cache that differ widely in size, or are not finite: the attention over the whole
cache and over a list, and a decode step, against the fp64 oracle, each 64 elements of a head by itself.

Tolerance: that of the 4-bit cache's other tests, with what a weight times its scale may lose counted per 64
elements: two fp16 terms hold it within 2^-22 of itself, or within 2^-31 of the largest such product of the
same 64 elements, which a code multiplies by 7 at most (so n 2^-31 of the largest weight times the largest
value of a row's 64 elements).
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from parity import tsl
from test_gpu_cache4 import Cache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _check(c, out, lse, b, tokens, spoilt=()):
    """out, lse of sequence b against the oracle; spoilt: (KV head, 64 elements) that have to be NaN throughout."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    d, n, scale = c.d, len(tokens), 1 / math.sqrt(c.d)
    for h in range(c.H):
        g = h // (c.H // c.Hkv)
        q = c.q[b, h].double().cpu().numpy()
        k, v = c.rows(c.kval, b, g, tokens), c.rows(c.vval, b, g, tokens)
        _, wl, w = O.attention(q, k, np.zeros_like(k), scale)
        el = scale * float(np.max(np.abs(k) @ np.abs(q) * (d + 16) * 2.0 ** -24
                                  + np.abs(k).sum(1) * np.abs(q).max() * 2.0 ** -21))
        assert abs(lse[b, h] - wl) <= el + n * 2.0 ** -23 + 2.0 ** -20 + abs(wl) * 2.0 ** -22
        for half in range(d // 64):
            e = slice(64 * half, 64 * half + 64)
            if (g, half) in spoilt:
                assert np.isnan(out[b, h, e]).all(), (b, h, half)
                continue
            want, mag = w @ v[:, e], w @ np.abs(v[:, e])
            big = n * float(np.max(w * np.abs(v[:, e]).max(1))) * 2.0 ** -31
            tol = mag * (2 * el + 2.0 ** -21 + 2.0 ** -20 + n * 2.0 ** -23) + big + 1e-30
            bad = np.abs(out[b, h, e] - want) / tol
            assert np.all(bad <= 1), (b, h, half, float(np.max(bad)), want[:2], out[b, h, e][:2])


def _write(c, k=None, v=None):
    c.ctx.append_prompt(c.k if k is None else k, c.v if v is None else v, c.cu, c.pt, c.kp, c.vp)
    c.kval, c.vval = (O.q4_pool_values(x.cpu().numpy(), c.d) for x in (c.kp, c.vp))


def _both(c, n):
    """Every token of the only sequence, through the whole-cache call and through a list."""
    out, lse = torch.zeros(1, c.H, c.d, device=DEV), torch.zeros(1, c.H, device=DEV)
    idx = torch.arange(n, dtype=torch.int32, device=DEV).view(1, n)
    for call in (lambda: c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out, lse),
                 lambda: c.ctx.sparse_attend(c.q, c.kp, c.vp, c.pt, idx, c.seq, out, lse)):
        out.zero_()
        lse.zero_()
        call()
        assert c.ctx.status() == 0
        yield out, lse


@pytest.mark.parametrize("H,Hkv", [(8, 2), (28, 4)])
@pytest.mark.parametrize("n", [16, 300, 2049])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_value_that_is_not_finite_spoils_its_own_64_elements_only(H, Hkv, n, bad):
    c = Cache(H, Hkv, 128, [n], seed=n + H)
    v = c.v.clone()
    v[3, 0, 70] = v[n - 1, 1, 5] = bad
    _write(c, v=v)
    for out, lse in _both(c, n):
        _check(c, out, lse, 0, np.arange(n), spoilt=((0, 1), (1, 0)))
    # a decode step, whose sinks and window hold both rows
    T = tsl()
    idx, cnt = torch.zeros(1, 84, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = torch.zeros(1, H, 128, device=DEV), torch.zeros(1, H, device=DEV)
    c.ctx.decode_step(c.q, c.kp, c.vp, c.pt, c.seq, T.params(k=64, n_sink=4, n_local=16), idx, cnt, out, lse)
    assert c.ctx.status() == 0
    _check(c, out, lse, 0, idx[0, :int(cnt[0])].cpu().numpy(), spoilt=((0, 1), (1, 0)))


@pytest.mark.parametrize("H,Hkv", [(8, 2), (28, 4)])
@pytest.mark.parametrize("n,at", [(64, 40), (700, 3), (16000, 8000)])
def test_a_large_value_costs_the_other_64_elements_nothing(H, Hkv, n, at):
    c = Cache(H, Hkv, 128, [n], seed=n + 1)
    v = c.v.clone()
    v[at, :, 64:] *= 2.0 ** 40
    _write(c, v=v)
    for out, lse in _both(c, n):
        _check(c, out, lse, 0, np.arange(n))


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (32, 8, 128), (28, 4, 128)])
@pytest.mark.parametrize("gap,small,large", [(110.0, 1.0, 1e30), (80.0, 1.0, 2000.0), (70.0, 1e-4, 2000.0), (55.0, 1e-9, 1e20),
                                             (30.0, 1e20, 1e-20)])
def test_logits_that_jump_far_between_pages(H, Hkv, d, gap, small, large):
    # the keys of half of the pages give logits `gap` below the others': the softmax has a new maximum in the first or
    # the second page of a warp's pair, and what came before counts for little or nothing
    n = 16000
    c = Cache(H, Hkv, d, [n], seed=5)
    # the heads share their query, 1.0 throughout; a key is its level in every element, and some noise
    c.q[:] = 1.0
    rng = np.random.default_rng(3)
    low = torch.from_numpy(np.repeat(rng.integers(0, 2, n // 16), 16)).to(DEV).view(n, 1, 1)
    k = (low * (-gap / math.sqrt(d)) + 0.05 * torch.randn(n, Hkv, d, device=DEV)).to(torch.bfloat16)
    _write(c, k=k, v=(c.v.float() * torch.where(low > 0, small, large)).to(torch.bfloat16))
    for out, lse in _both(c, n):
        assert torch.isfinite(out).all()
        _check(c, out, lse, 0, np.arange(n))


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (32, 8, 128), (28, 4, 128)])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-8, 1e-20, 1e6])
def test_pages_of_zero_values_among_others(H, Hkv, d, size):
    # half of the pages have value rows of zeros, the first among them
    n = 16000
    c = Cache(H, Hkv, d, [n], seed=6)
    rng = np.random.default_rng(4)
    keep = np.repeat(rng.integers(0, 2, n // 16), 16)
    keep[:16] = 0
    v = c.v.float() * size * torch.from_numpy(keep).to(DEV).view(n, 1, 1)
    _write(c, v=v.to(torch.bfloat16))
    for out, lse in _both(c, n):
        _check(c, out, lse, 0, np.arange(n))


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (28, 4, 128)])
def test_a_first_page_of_zero_values_in_a_short_sequence(H, Hkv, d):
    c = Cache(H, Hkv, d, [64], seed=7)
    v = c.v.float() * 1e-6
    v[:16] = 0
    _write(c, v=v.to(torch.bfloat16))
    for out, lse in _both(c, 64):
        _check(c, out, lse, 0, np.arange(64))


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (32, 8, 128), (28, 4, 128)])
@pytest.mark.parametrize("n,cut", [(64, 48), (2000, 1000), (9000, 8990)])
def test_logits_that_leave_fp32_weigh_nothing_beside_finite_ones(H, Hkv, d, n, cut):
    # the first `cut` keys give logits near -1e39, which fp32 holds as -inf; the others give 0 throughout, so the
    # weights are 0 and 1 / (n - cut)
    c = Cache(H, Hkv, d, [n], seed=8)
    c.q[:] = 0
    c.q[:, :, 0] = 1e20
    k = torch.zeros_like(c.k)
    k[:cut, :, 0] = -1e20
    _write(c, k=k)
    rest = n - cut
    for out, lse in _both(c, n):
        for h in range(H):
            v = c.rows(c.vval, 0, h // (H // Hkv), np.arange(cut, n))
            tol = np.abs(v).mean(0) * (2.0 ** -21 + 2.0 ** -20 + n * 2.0 ** -23) + np.abs(v).max() * n * 2.0 ** -31
            assert np.all(np.abs(out[0, h].double().cpu().numpy() - v.mean(0)) <= tol)
        assert torch.all(torch.abs(lse.double() - math.log(rest)) <= n * 2.0 ** -23 + 2.0 ** -20 + math.log(rest) * 2.0 ** -22)
    vote = torch.full((1, c.ctx.max_tokens), 7.0, device=DEV)
    c.ctx.score(c.q, c.kp, c.pt, c.seq, vote)
    assert c.ctx.status() == 0
    assert not vote[0, :cut].any()
    assert torch.all(torch.abs(vote[0, cut:n].double() * rest / H - 1) <= n * 2.0 ** -23 + 2.0 ** -19)


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (28, 4, 128)])
def test_a_sequence_without_a_page_in_the_pool_has_votes_of_zero(H, Hkv, d):
    T = tsl()
    c = Cache(H, Hkv, d, [100, 300], seed=9)
    ref, vote = (torch.full((2, c.ctx.max_tokens), 7.0, device=DEV) for _ in range(2))
    c.ctx.score(c.q, c.kp, c.pt, c.seq, ref)
    assert c.ctx.status() == 0
    bad = c.pt.clone()
    bad[0] = c.pages
    c.ctx.score(c.q, c.kp, bad, c.seq, vote)
    assert c.ctx.status() == T.STATUS_CODE["TS_ERR_PAGE_OOB"]
    assert not vote[0, :100].any() and torch.equal(vote[1], ref[1]) and (vote[0, 100:] == 7).all()
    # a decode step over it: the lowest candidates (all votes are equal), and no token to attend to
    idx, cnt = torch.zeros(2, 30, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    out, lse = torch.ones(2, H, d, device=DEV), torch.ones(2, H, device=DEV)
    c.ctx.decode_step(c.q, c.kp, c.vp, bad, c.seq, T.params(k=10, n_sink=4, n_local=16), idx, cnt, out, lse)
    assert c.ctx.status() == T.STATUS_CODE["TS_ERR_PAGE_OOB"]
    assert idx[0].tolist() == list(range(14)) + list(range(84, 100)) and cnt.tolist() == [30, 30]
    assert not out[0].any() and torch.isinf(lse[0]).all() and torch.isfinite(out[1]).all()


def test_queries_and_rows_of_another_type_are_refused():
    T = tsl()
    c = Cache(8, 2, 128, [100, 30], seed=10)
    out, lse = torch.full((2, 8, 128), 7.0, device=DEV), torch.full((2, 8), 7.0, device=DEV)
    idx, cnt = torch.zeros(2, 30, dtype=torch.int32, device=DEV), torch.full((2,), 3, dtype=torch.int32, device=DEV)
    kn = torch.ones(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    kp = c.kp.clone()
    q = c.q.to(torch.bfloat16)
    for call in (lambda: c.ctx.attend(q, c.kp, c.vp, c.pt, c.seq, out, lse),
                 lambda: c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq.long(), out, lse),
                 lambda: c.ctx.attend(c.q, c.kp, c.vp, c.pt[:, :-1].contiguous(), c.seq, out, lse),
                 lambda: c.ctx.attend(c.q, c.kp[:-1], c.vp, c.pt, c.seq, out, lse),
                 lambda: c.ctx.attend(c.q, c.kp, c.vp, c.pt, c.seq, out.to(torch.bfloat16), lse),
                 lambda: c.ctx.sparse_attend(q, c.kp, c.vp, c.pt, idx, cnt, out, lse),
                 lambda: c.ctx.decode_step(q, c.kp, c.vp, c.pt, c.seq, T.params(), idx, cnt, out, lse),
                 lambda: c.ctx.score(q, c.kp, c.pt, c.seq, torch.zeros(2, c.ctx.max_tokens, device=DEV)),
                 lambda: c.ctx.append_kv(kn.float(), kn, c.pt, c.seq, c.kp, c.vp),
                 lambda: c.ctx.append_kv(kn[:1], kn, c.pt, c.seq, c.kp, c.vp),
                 lambda: c.ctx.append_prompt(c.k, c.v, c.cu, c.pt[:1], c.kp, c.vp),
                 lambda: c.ctx.read_kv(c.cu, c.pt, c.kp[:-1], c.vp, *(torch.zeros(130, 2, 128, device=DEV) for _ in range(2)))):
        with pytest.raises(T.TokenSelectError):
            call()
    assert (out == 7).all() and (lse == 7).all() and torch.equal(c.kp, kp) and c.ctx.status() == 0


def test_a_context_for_many_prompts_holds_no_scratch_of_other_kernels():
    # 531 sequences of 32 heads over 8: the parts of the kernels that do not serve 4-bit pools would be 1.9 GB
    T = tsl()
    T.Context(32, 8, 128, T.TS_KV_Q4, 1, 1, 1).close()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    ctx = T.Context(32, 8, 128, T.TS_KV_Q4, 531, 1, 1)
    held = free - torch.cuda.mem_get_info()[0]
    ctx.close()
    assert held < 256 << 20, held


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (32, 8, 128), (28, 4, 128)])
def test_from_prompts_to_decode_steps_within_each_operator_s_tolerance(H, Hkv, d):
    # prompts are attended and written, then decode steps append, select and attend: every output against the oracle
    # over the values that the cache holds, as near as the operators by themselves
    from test_gpu_prompt import _check as check_prompt
    T = tsl()
    lens, steps = [333, 1, 70], 3
    B, rows = len(lens), sum(lens)
    c = Cache(H, Hkv, d, [n + steps for n in lens], seed=22, poison=False)
    c.kp.fill_(255)                                                # (slots not written yet hold NaN)
    c.vp.fill_(255)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    qkv = torch.randn(rows, (H + 2 * Hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
    q = qkv[:, :H * d].view(rows, H, d)
    k, v = (qkv[:, (H + i * Hkv) * d:(H + (i + 1) * Hkv) * d].view(rows, Hkv, d) for i in range(2))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu_dev = torch.from_numpy(cu).to(DEV)
    out, lse = torch.zeros(rows, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, H, device=DEV)
    c.ctx.prompt_attend(q, k, v, cu_dev, out, lse)
    c.ctx.append_prompt(k, v, cu_dev, c.pt, c.kp, c.vp)
    assert c.ctx.status() == 0
    check_prompt(out, lse, q, k, v, cu, 1 / math.sqrt(d), [0, 1, 127, 128, 255, 256, 332, 333, 334, 403])
    cache, prm = c.ctx.cache(1, 52), T.params(k=32, n_sink=4, n_local=16, theta=0.9)
    idx, cnt = torch.zeros(B, 52, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    o, z, full, fullz = (torch.zeros(B, H, *x, device=DEV) for x in ((d,), (), (d,), ()))
    hit = torch.zeros(B, dtype=torch.uint8, device=DEV)
    states, hits = [O.CacheState() for _ in range(B)], 0
    for t in range(steps):
        seq = torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device=DEV)
        kn, vn = (torch.randn(B, Hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        noise = torch.randn(B, H, d, generator=g, device=DEV)
        c.q = noise if t != 1 else c.q + 0.1 * noise
        c.ctx.append_kv(kn, vn, c.pt, seq, c.kp, c.vp)
        c.ctx.decode_step(c.q, c.kp, c.vp, c.pt, seq, prm, idx, cnt, o, z, hit=hit, cache=cache)
        c.ctx.attend(c.q, c.kp, c.vp, c.pt, seq, full, fullz)
        assert c.ctx.status() == 0
        c.kval, c.vval = (O.q4_pool_values(x.cpu().numpy(), d) for x in (c.kp, c.vp))
        for b in range(B):
            n = lens[b] + t + 1
            ref = O.decode_step(states[b], c.q[b].double().cpu().numpy(), c.kval, c.vval, c.table[b], n, k=32, n_sink=4,
                                n_local=16, theta=0.9)
            got = idx[b, :int(cnt[b])].cpu().numpy()
            assert bool(hit[b]) == ref["hit"] and np.array_equal(got, ref["idx"])
            hits += ref["hit"]
            _check(c, o, z, b, got)
            _check(c, full, fullz, b, np.arange(n))
    assert hits == B


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (28, 4, 128)])
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_values_at_the_end_of_fp32_s_range(H, Hkv, d, n):
    # every value is near 3e38: the outputs are finite, the sums of weights times values are not
    c = Cache(H, Hkv, d, [n], seed=11)
    _write(c, v=(3e38 * (1 - 0.1 * torch.rand(n, Hkv, d, device=DEV))).to(torch.bfloat16))
    for out, lse in _both(c, n):
        _check(c, out, lse, 0, np.arange(n))
