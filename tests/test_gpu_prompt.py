"""ts_prompt_attend on the GPU against the fp64 oracle: ragged packed prompts, grouped heads, strides,
and masked places that hold NaN or infinities.

Tolerance, per row with weights w and values v: a score is a sum of d products that are exact in fp32,
off by el = alpha sum|q_e k_e| (d + 16) 2^-24, and its exponential by 2^-20; a weight is rounded to
bf16 for its product (2^-8), sums of n terms are off by n 2^-23, the output is rounded to bf16 (2^-8).
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _make(H, Hkv, d, lens, seed=0, spread=1.5, extra=0):
    """q, k, v as column ranges of one matrix, `extra` rows behind the last sequence."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows = sum(lens) + extra
    m = torch.randn(rows, (H + 2 * Hkv) * d, generator=g, device=DEV)
    m[:, :H * d] *= spread
    m = m.to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return (m[:, :H * d].view(rows, H, d), m[:, H * d:(H + Hkv) * d].view(rows, Hkv, d),
            m[:, (H + Hkv) * d:].view(rows, Hkv, d), torch.from_numpy(cu).to(DEV), cu)


def _ctx(H, Hkv, d, B):
    T = tsl()
    return T.Context(H, Hkv, d, T.TS_KV_Q4, B, 1, 1)


def _check(out, lse, q, k, v, cu, scale, rows=None):
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    H, d = q.shape[1:]
    group = H // k.shape[1]
    worst = 0.0
    for lo, hi in zip(cu[:-1], cu[1:]):
        for r in range(lo, hi) if rows is None else [x for x in rows if lo <= x < hi]:
            for h in range(H):
                kk, vv = k[lo:r + 1, h // group], v[lo:r + 1, h // group]
                want, wl, w = O.attention(q[r, h], kk, vv, scale)
                el = abs(scale) * float(np.max(np.abs(kk) @ np.abs(q[r, h]))) * (d + 16) * 2.0 ** -24
                n = r + 1 - lo
                tol = (w @ np.abs(vv)) * (2.0 ** -8 + 2 * el + 2.0 ** -20 + n * 2.0 ** -23) + np.abs(want) * 2.0 ** -8
                worst = max(worst, float(np.max(np.abs(out[r, h] - want) / (tol + 1e-30))))
                assert np.all(np.abs(out[r, h] - want) <= tol + 1e-30), (r, h, worst)
                assert abs(lse[r, h] - wl) <= el + n * 2.0 ** -23 + 2.0 ** -20 + abs(wl) * 2.0 ** -22
    return worst


GEOS = [(1, 1, 64), (4, 4, 128), (8, 4, 64), (32, 8, 128), (28, 4, 128), (5, 1, 64), (16, 1, 128), (24, 2, 64)]


@pytest.mark.parametrize("H,Hkv,d", GEOS)
@pytest.mark.parametrize("lens", [[1], [0, 3, 129, 0, 128, 17], [300]])
def test_prompts_against_the_oracle(H, Hkv, d, lens):
    q, k, v, cu_dev, cu = _make(H, Hkv, d, lens, seed=H + d + len(lens), extra=2)
    rows = q.shape[0]
    out = torch.full((rows, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows, H), 7.0, device=DEV)
    ctx = _ctx(H, Hkv, d, len(lens))
    ctx.prompt_attend(q, k, v, cu_dev, out, lse)
    assert ctx.status() == 0
    _check(out, lse, q, k, v, cu, 1 / math.sqrt(d))
    assert (out[cu[-1]:] == 7).all() and (lse[cu[-1]:] == 7).all()
    # again without lse, into a strided output: the same bits, and nothing beside the rows
    wide = torch.full((rows, H * d + 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ctx.prompt_attend(q, k, v, cu_dev, wide[:, :H * d].view(rows, H, d))
    assert torch.equal(wide[:, :H * d].reshape(rows, H, d), out) and (wide[:, H * d:] == 7).all()


@pytest.mark.parametrize("H,Hkv,d,n", [(8, 8, 128, 1000), (28, 4, 128, 1500), (8, 4, 64, 2100)])
def test_longer_prompts_at_tile_borders(H, Hkv, d, n):
    q, k, v, cu_dev, cu = _make(H, Hkv, d, [n, 700], seed=n)
    out, lse = torch.zeros(n + 700, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n + 700, H, device=DEV)
    ctx = _ctx(H, Hkv, d, 2)
    ctx.prompt_attend(q, k, v, cu_dev, out, lse)
    assert ctx.status() == 0
    t = 2 * (128 // (H // Hkv))
    rows = sorted({r for base in (0, n) for m in (1, 2, 3, 5) for r in (base + m * t - 1, base + m * t, base + 128 * m - 1, base + 128 * m)}
                  | {0, n - 1, n, n + 699})
    _check(out, lse, q, k, v, cu, 1 / math.sqrt(d), [r for r in rows if r < n + 700])


@pytest.mark.parametrize("scale", [-0.2, 0.5, 1e-3])
def test_scales_and_maxima_that_move(scale):
    # the keys grow along the prompt, so the running maximum of late rows moves in every tile
    H, Hkv, d, n = 4, 2, 64, 700
    q, k, v, cu_dev, cu = _make(H, Hkv, d, [n], seed=3)
    k = (k.float() * torch.linspace(0.05, 8.0, n, device=DEV).view(-1, 1, 1)).to(torch.bfloat16)
    out, lse = torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n, H, device=DEV)
    ctx = _ctx(H, Hkv, d, 1)
    ctx.prompt_attend(q, k, v, cu_dev, out, lse, scale=scale)
    _check(out, lse, q, k, v, cu, scale, [0, 1, 63, 64, 127, 128, 300, 512, 699])


@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (7, 1, 64), (4, 4, 128)])
def test_no_row_sees_what_is_masked(H, Hkv, d):
    # every row of k and v from `cut` on, of another sequence or past the end, holds NaN or infinities
    lens, extra = [70, 150, 400], 40
    q, k, v, cu_dev, cu = _make(H, Hkv, d, lens, seed=11, extra=extra)
    ctx = _ctx(H, Hkv, d, 3)
    rows = q.shape[0]
    base = torch.zeros(rows, H, d, dtype=torch.bfloat16, device=DEV)
    base_lse = torch.zeros(rows, H, device=DEV)
    ctx.prompt_attend(q, k, v, cu_dev, base, base_lse)
    for bad in (float("nan"), float("inf"), float("-inf")):
        for seq, cut in ((0, 33), (1, 0), (1, 149), (2, 257), (2, 128), (2, 400)):
            kk, vv = k.clone(), v.clone()
            lo, hi = cu[seq] + cut, (cu[seq + 1] if cut < lens[seq] else rows)
            kk[lo:hi], vv[lo:hi] = bad, bad
            out, lse = torch.zeros_like(base), torch.zeros_like(base_lse)
            ctx.prompt_attend(q, kk, vv, cu_dev, out, lse)
            keep = torch.ones(rows, dtype=torch.bool, device=DEV)
            keep[lo:hi] = False
            assert torch.equal(out[keep], base[keep]) and torch.equal(lse[keep], base_lse[keep]), (bad, seq, cut)
            if cut < lens[seq] and bad != bad:
                assert torch.isnan(out[lo:hi]).all()


def test_values_that_are_not_finite_reach_the_rows_that_see_them():
    H, Hkv, d, n = 8, 2, 128, 200
    q, k, v, cu_dev, cu = _make(H, Hkv, d, [n], seed=13)
    ctx = _ctx(H, Hkv, d, 1)
    base, out = (torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ctx.prompt_attend(q, k, v, cu_dev, base)
    v = v.clone()
    v[150, 0, 5], v[160, 0, 5] = float("inf"), float("-inf")       # inf, then NaN from 160 on
    v[170, 0, 100] = float("nan")
    v[20, 1, 7] = float("-inf")
    ctx.prompt_attend(q, k, v, cu_dev, out)
    want = base.clone().float()
    want[150:160, :4, 5] = float("inf")
    want[160:, :4, 5] = float("nan")
    want[170:, :4, 100] = float("nan")
    want[20:, 4:, 7] = float("-inf")
    assert torch.equal(torch.nan_to_num(out.float(), 123.0), torch.nan_to_num(want, 123.0))


def test_a_nan_query_stays_in_its_row():
    H, Hkv, d, n = 28, 4, 128, 90
    q, k, v, cu_dev, cu = _make(H, Hkv, d, [n], seed=17)
    ctx = _ctx(H, Hkv, d, 1)
    base, out = (torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ctx.prompt_attend(q, k, v, cu_dev, base)
    q = q.clone()
    q[40, 9, 3] = float("nan")
    ctx.prompt_attend(q, k, v, cu_dev, out)
    assert torch.isnan(out[40, 9]).all()
    out[40, 9] = base[40, 9]
    assert torch.equal(out, base)


def test_the_same_bits_again_and_in_a_graph_and_in_any_packing():
    H, Hkv, d = 28, 4, 128
    lens = [257, 1, 700, 33, 90]
    q, k, v, cu_dev, cu = _make(H, Hkv, d, lens, seed=19)
    ctx = _ctx(H, Hkv, d, 40)
    n = sum(lens)
    out = torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV)
    ctx.prompt_attend(q, k, v, cu_dev, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = torch.zeros_like(out)
    with torch.cuda.stream(s):
        ctx.prompt_attend(q, k, v, cu_dev, again)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ctx.prompt_attend(q, k, v, cu_dev, again)
        again.zero_()
        for _ in range(20):
            g.replay()
    s.synchronize()
    assert torch.equal(out, again)
    # each prompt alone, and among many empty ones
    for b, x in enumerate(lens):
        lo = cu[b]
        alone = torch.zeros(x, H, d, dtype=torch.bfloat16, device=DEV)
        ctx.prompt_attend(q[lo:lo + x], k[lo:lo + x], v[lo:lo + x],
                          torch.tensor([0] * 17 + [x] * 3, dtype=torch.int32, device=DEV), alone)
        assert torch.equal(alone, out[lo:lo + x])
    # forty sequences: more than a warp has lanes
    many = torch.tensor(list(range(0, 39 * 28, 28)) + [n - 5, n], dtype=torch.int32, device=DEV)[:41]
    lens40 = (many[1:] - many[:-1]).tolist()
    assert min(lens40) >= 0 and sum(lens40) <= n
    out40, lse40 = torch.zeros_like(out), torch.zeros(n, H, device=DEV)
    ctx.prompt_attend(q, k, v, many, out40, lse40)
    assert ctx.status() == 0
    _check(out40, lse40, q, k, v, many.tolist(), 1 / math.sqrt(d), [0, 27, 28, 500, 39 * 28 - 30, n - 6, n - 5, n - 1])


def test_scores_of_minus_infinity_in_the_first_tiles():
    # every key but the last 30 gives -inf for head 0 (its queries point against an infinite key element), so
    # the rows behind them see their first finite score late; rows that see none are NaN, as a softmax over
    # nothing but -inf is
    H, Hkv, d, n, cut = 2, 1, 64, 400, 370
    q, k, v, cu_dev, cu = _make(H, Hkv, d, [n], seed=37, spread=0.1)
    q, k = q.clone(), k.clone()
    q[:, 0, 0], q[:, 1, 0] = -1.0, -2.0
    k[:cut, 0, 0] = float("inf")
    out, lse = torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n, H, device=DEV)
    ctx = _ctx(H, Hkv, d, 1)
    ctx.prompt_attend(q, k, v, cu_dev, out, lse)
    assert torch.isnan(out[:cut]).all()
    alone, alone_lse = torch.zeros(n - cut, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n - cut, H, device=DEV)
    ctx.prompt_attend(q[cut:], k[cut:], v[cut:], torch.tensor([0, n - cut], dtype=torch.int32, device=DEV), alone, alone_lse)
    # the same weights over the same rows; sums in another grouping, outputs rounded to bf16
    assert torch.allclose(lse[cut:], alone_lse, rtol=0, atol=2.0 ** -18)
    assert torch.allclose(out[cut:].float(), alone.float(), rtol=2.0 ** -7, atol=2.0 ** -7)


def test_three_hundred_prompts_at_once():
    H, Hkv, d = 8, 2, 64
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.choice([0, 1, 3, 20, 63, 64, 65, 140], 300)]
    q, k, v, cu_dev, cu = _make(H, Hkv, d, lens, seed=31)
    n = sum(lens)
    out, lse = torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n, H, device=DEV)
    ctx = _ctx(H, Hkv, d, 300)
    ctx.prompt_attend(q, k, v, cu_dev, out, lse)
    assert ctx.status() == 0
    rows = {0, n - 1} | {int(cu[b]) for b in range(0, 300, 13) if lens[b]} | {int(cu[b + 1]) - 1 for b in range(0, 300, 13) if lens[b]}
    _check(out, lse, q, k, v, cu, 1 / math.sqrt(d), sorted(rows))


def test_rows_past_four_gigabytes():
    # the last prompt lies behind 2^31 elements of q and out: the same bits as by itself
    H, Hkv, d, n, many = 32, 8, 128, 333, 530
    q, k, v, cu1, _ = _make(H, Hkv, d, [n], seed=12)
    rows = many * 1000 + n
    cu = torch.tensor([1000 * i for i in range(many + 1)] + [rows], dtype=torch.int32, device=DEV)
    big = [torch.zeros(rows, x.shape[1], d, dtype=torch.bfloat16, device=DEV) for x in (q, k, v)]
    assert (rows - n) * H * d > 1 << 31
    for x, y in zip(big, (q, k, v)):
        x[-n:] = y
    out, lse = torch.zeros(rows, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, H, device=DEV)
    ctx = _ctx(H, Hkv, d, many + 1)
    ctx.prompt_attend(*big, cu, out, lse)
    out1, lse1 = torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n, H, device=DEV)
    ctx.prompt_attend(q, k, v, cu1, out1, lse1)
    assert ctx.status() == 0
    assert torch.equal(out[-n:], out1) and torch.equal(lse[-n:], lse1)
    assert not out[:-n].any()


def test_bad_boundaries_are_reported_and_nothing_else_is_written():
    T = tsl()
    H, Hkv, d = 8, 4, 64
    q, k, v, _, _ = _make(H, Hkv, d, [100], seed=23)
    ctx = _ctx(H, Hkv, d, 3)
    SEQ = T.STATUS_CODE["TS_ERR_SEQ_LEN"]
    good = torch.zeros(100, H, d, dtype=torch.bfloat16, device=DEV)
    ctx.prompt_attend(q, k, v, torch.tensor([0, 40, 40, 100], dtype=torch.int32, device=DEV), good)
    assert ctx.status() == 0
    for cu, first in (([0, 40, 40, 101], 40), ([0, 40, 20, 10], 40), ([0, 40, -5, -9], 40)):
        out = torch.full_like(good, 7.0)
        ctx.prompt_attend(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), out)
        assert ctx.status() == SEQ
        assert torch.equal(out[:first], good[:first]) and (out[first:] == 7).all()
    out = torch.full_like(good, 7.0)
    ctx.prompt_attend(q, k, v, torch.tensor([0, 40, 40, 100], dtype=torch.int32, device=DEV), out)
    assert ctx.status() == 0 and torch.equal(out, good)


def test_refusals():
    T = tsl()
    H, Hkv, d = 8, 4, 64
    q, k, v, cu, _ = _make(H, Hkv, d, [10], seed=29)
    out = torch.zeros(10, H, d, dtype=torch.bfloat16, device=DEV)
    ctx = _ctx(H, Hkv, d, 1)

    def refused(code, c, *a):
        with pytest.raises(T.TokenSelectError) as e:
            T.ts_prompt_attend(c.handle, *a)
        assert e.value.status == T.STATUS_CODE[code]

    st, qs = q.stride(0), H * d
    refused("TS_ERR_UNSUPPORTED", T.Context(8, 2, 64, T.TS_KV_F32, 1, 1, 1), q, st, k, st, v, st, cu, 1, 10, 0.0, out, qs)
    refused("TS_ERR_INVALID_ARG", ctx, q, st, k, st, v, st, cu, 1, 10, float("nan"), out, qs)
    refused("TS_ERR_INVALID_ARG", ctx, q, st, k, st, v, st, None, 1, 10, 0.0, out, qs)
    refused("TS_ERR_INVALID_ARG", ctx, q.data_ptr() + 2, st, k, st, v, st, cu, 1, 10, 0.0, out, qs)
    refused("TS_ERR_INVALID_ARG", ctx, q, st, k, st + 4, v, st, cu, 1, 10, 0.0, out, qs)
    refused("TS_ERR_SHAPE", ctx, q, st, k, st, v, st, cu, 1, 10, 0.0, out, qs - 8)
    refused("TS_ERR_SHAPE", ctx, q, st, k, 1 << 40, v, st, cu, 1, 10, 0.0, out, qs)
    refused("TS_ERR_SHAPE", ctx, q, st, k, st, v, st, cu, 2, 10, 0.0, out, qs)
    refused("TS_ERR_SHAPE", ctx, q, st, k, st, v, st, cu, 0, 10, 0.0, out, qs)
    refused("TS_ERR_SHAPE", ctx, q, st, k, st, v, st, cu, 1, -1, 0.0, out, qs)
    for bad in (dict(k=k[:9]), dict(v=v[:, :2]), dict(out=out[:9]), dict(lse=torch.zeros(10, H, dtype=torch.bfloat16, device=DEV)),
                dict(q=q.float()), dict(out=out.float()), dict(cu=cu.long()), dict(k=k.cpu()),
                dict(lse=torch.zeros(10, 2 * H, device=DEV)[:, :H])):
        a = dict(dict(q=q, k=k, v=v, cu=cu, out=out, lse=None), **bad)
        with pytest.raises(T.TokenSelectError):
            ctx.prompt_attend(a["q"], a["k"], a["v"], a["cu"], a["out"], a["lse"])
    T.ts_prompt_attend(ctx.handle, q, st, k, st, v, st, cu, 1, 0, 0.0, out, qs)                  # no rows: nothing to do
    assert not out.any() and ctx.status() == 0
