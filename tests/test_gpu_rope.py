"""ts_rotate and ts_append_rotated on the GPU against the rational-angle oracle.

Tolerance of a turned element, a (x1 cos - x2 sin): the angle in half turns is rounded to fp32 (2^-25 of one, so pi
2^-25 < 1.6 2^-24 radians) after 2^-32 of a turn is cut off (0.03 2^-24), cos and sin are right to 2 ulps (2 2^-24), their product
with a, the two products and the sum round (a half ulp each: at most 4 2^-24 of |x1| + |x2|): below 8 2^-24 a (|x1| + |x2|) in all;
then the output's own rounding, eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import draft_oracle as D
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
KIND = {"bf16": BF, "fp32": F32}

PLAIN = dict(base=10000.0)
BANDS = dict(base=500000.0, scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0)
YARN = dict(base=10000.0, scaling="yarn", factor=4.0, original=4096, low=1.0, high=32.0)
LINEAR = dict(base=10000.0, scaling="linear", factor=2.0)


def _rows(rows, heads, d, kind, seed, extra=64):
    """[rows][heads][d] cut from wider rows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    m = torch.randn(rows, heads * d + extra, generator=g, device=DEV).to(kind)
    return m[:, :heads * d].view(rows, heads, d) if rows else m[:, :heads * d].reshape(0, heads, d)


def _check(got, x, positions, rope, r, pairs):
    f, a = rope.read()
    x, got_ = x.double().cpu().numpy(), got.double().cpu().numpy()
    want = D.rotate(x, positions, f, a, r, pairs)
    size = np.zeros_like(want)
    h = r // 2
    i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if pairs else (np.arange(h), np.arange(h, r))
    both = np.abs(x[..., i]) + np.abs(x[..., j])
    size[..., i] = size[..., j] = both
    tol = 8 * 2.0 ** -24 * a * size + np.abs(want) * torch.finfo(got.dtype).eps / 2 * (1 + 2.0 ** -10)
    assert np.all(np.abs(got_ - want) <= tol), np.max(np.abs(got_ - want) / np.maximum(tol, 1e-300))
    if r < x.shape[-1]:
        assert np.array_equal(got_[..., r:], torch.from_numpy(x[..., r:]).to(got.dtype).double().numpy())


@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("d,r,pairs,cfg", [
    (128, 128, False, PLAIN), (128, 128, True, BANDS), (128, 64, False, YARN), (128, 2, False, PLAIN), (128, 6, True, LINEAR),
    (64, 64, False, LINEAR), (64, 32, True, YARN), (64, 48, False, BANDS), (64, 36, False, PLAIN), (128, 126, False, YARN),
    (64, 2, True, PLAIN), (128, 16, False, PLAIN)])
def test_rows_against_the_oracle(d, r, pairs, cfg, src, dst):
    T = tsl()
    ctx = T.Context(8, 8, d, T.TS_KV_Q4, 1, 1, 1)
    rope = ctx.rope(r, interleaved=pairs, **cfg)
    for rows, heads in ((1, 3), (7, 8), (611, 1)):
        x = _rows(rows, heads, d, KIND[src], rows)
        rng = np.random.default_rng(rows)
        pos = rng.integers(0, 131072, rows)
        pos[:2] = [0, 2 ** 31 - 1][:rows]
        pos[-1] = 1000003
        if rows > 4:
            pos[3:5] = [-5, -2 ** 31]
        out = torch.full((rows, heads, d), 7.0, dtype=KIND[dst], device=DEV)
        ctx.rotate(rope, x, torch.from_numpy(pos.astype(np.int32)).to(DEV), out)
        assert ctx.status() == 0
        _check(out, x, pos, rope, r, pairs)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("d,r,pairs", [(128, 128, False), (64, 36, False), (128, 128, True), (64, 48, False)])
def test_in_place_gives_the_same_bits(d, r, pairs, kind):
    T = tsl()
    ctx = T.Context(8, 8, d, T.TS_KV_Q4, 1, 1, 1)
    rope = ctx.rope(r, interleaved=pairs)
    x = _rows(1301, 5, d, KIND[kind], 4)
    pos = torch.arange(1301, dtype=torch.int32, device=DEV) * 977
    out = torch.empty_like(x)
    ctx.rotate(rope, x, pos, out)
    ctx.rotate(rope, x, pos, x)
    assert torch.equal(out, x)


def test_negated_positions_are_the_transpose_and_the_gradient():
    """<g, R x> = <R^T g, x>, and differences of <g, R x> along every element of a head give R^T g."""
    T = tsl()
    d, r = 64, 48
    ctx = T.Context(4, 4, d, T.TS_KV_Q4, 1, 1, 1)
    rope = ctx.rope(r, **YARN)
    pos = torch.tensor([0, 3, 500, 131071, -9], dtype=torch.int32, device=DEV)
    x, g = _rows(5, 2, d, F32, 1), _rows(5, 2, d, F32, 2)
    y, gx = torch.empty(5, 2, d, device=DEV), torch.empty(5, 2, d, device=DEV)
    ctx.rotate(rope, x, pos, y)
    ctx.rotate(rope, g, -pos, gx)
    lhs, rhs = (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
    size = float(g.double().abs().sum() * x.double().abs().max())
    assert abs(float(lhs - rhs)) <= size * 16 * 2.0 ** -24 * rope.read()[1]
    # the map is linear: R (x + e) - R x for unit steps, both exact to the rounding of their elements
    f, a = rope.read()
    for e in range(d):
        step = x.clone()
        step[..., e] += 1.0
        y1 = torch.empty_like(y)
        ctx.rotate(rope, step, pos, y1)
        diff = ((y1.double() - y.double()) * g.double()).sum(-1)
        # y1 - y: 8 2^-24 a (|x1| + |x2|) and a rounding of either, in the (at most) two elements of the pair
        lim = 40 * 2.0 ** -24 * a * (x.double().abs().amax(-1) + 2) * g.double().abs().amax(-1)
        assert torch.all((diff - gx[..., e].double()).abs() <= lim), e


def test_what_is_not_turned_and_not_finite():
    """Elements behind r keep their bits (NaN, -0 too), a NaN stays in its own pair, rows behind `total` stay."""
    T = tsl()
    for d, r, pairs in ((64, 32, False), (64, 36, False), (64, 36, True)):
        ctx = T.Context(4, 4, d, T.TS_KV_Q4, 1, 1, 1)
        rope = ctx.rope(r, interleaved=pairs)
        buf = _rows(6, 2, d, F32, 3)
        buf[..., r:] = -0.0
        buf[1, 0, r] = float("nan")
        buf[2, 1, d - 1] = float("-inf")
        buf[3, 0, 0] = float("inf")
        x = buf[:5]
        out = torch.full((6, 2, d), 5.0, device=DEV)
        ctx.rotate(rope, x, torch.arange(1, 6, dtype=torch.int32, device=DEV), out[:5])
        assert torch.all(out[5] == 5.0)
        same = out[:5, :, r:].contiguous().view(torch.int32) == x[..., r:].contiguous().view(torch.int32)
        assert bool(same.all())
        bad = ~torch.isfinite(out[:5])
        partner = 1 if pairs else r // 2
        want = torch.zeros_like(bad)
        want[1, 0, r] = want[2, 1, d - 1] = want[3, 0, 0] = want[3, 0, partner] = True
        assert torch.equal(bad, want)


def test_given_frequencies_and_a_factor():
    """Any frequencies: more than a turn per position, backwards, tiny, zero."""
    T = tsl()
    ctx = T.Context(4, 4, 64, T.TS_KV_Q4, 1, 1, 1)
    rope = ctx.rope(12, scaling="given", freqs=[1.0, -0.25, 7.5, 1234.5678, 3e-9, 0.0], attention=0.75)
    for pairs in (False, True):
        rope = ctx.rope(12, interleaved=pairs, scaling="given", freqs=[1.0, -0.25, 7.5, 1234.5678, 3e-9, 0.0], attention=0.75)
        x = _rows(9, 2, 64, F32, 8)
        pos = np.array([0, 1, 5, 77, 131071, 10 ** 6, 2 ** 31 - 1, -1, -2 ** 31])
        out = torch.empty(9, 2, 64, device=DEV)
        ctx.rotate(rope, x, torch.from_numpy(pos.astype(np.int32)).to(DEV), out)
        assert ctx.status() == 0
        _check(out, x, pos, rope, 12, pairs)


def test_no_rows_is_nothing_to_do():
    T = tsl()
    ctx = T.Context(4, 4, 64, T.TS_KV_Q4, 1, 1, 1)
    rope = ctx.rope()
    n = ctx.rotate(rope, _rows(0, 2, 64, F32, 0), torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(0, 2, 64, device=DEV))
    assert n is None and T.ts_kernel_count(ctx.handle) == 0


# ------------------------------------------------------------ into the pools

POOLS = [("bf16", 8, 4, 128, 16), ("bf16", 4, 2, 64, 16), ("bf16", 4, 7, 128, 16), ("bf16", 8, 1, 128, 1), ("fp32", 8, 4, 128, 16),
         ("fp32", 2, 4, 64, 16), ("fp32", 4, 1, 64, 1), ("4bit", 3, 2, 128, 16), ("4bit", 1, 5, 64, 16)]


def _context(T, kv, HKV, G, d, page, B, max_pages, pages):
    t = {"bf16": T.TS_KV_BF16, "fp32": T.TS_KV_F32, "4bit": T.TS_KV_Q4}[kv]
    return T.Context(HKV * G, HKV, d, t, B, max_pages, pages, page)


def _pool(kv, pages, HKV, page, d):
    if kv == "4bit":
        return torch.full((pages, HKV, 16 * (d // 2 + d // 32)), 0x5a, dtype=torch.uint8, device=DEV)
    return torch.full((pages, HKV, page, d), 3.0, dtype=KIND[kv], device=DEV)


@pytest.mark.parametrize("kv,HKV,G,d,page", POOLS)
@pytest.mark.parametrize("lens", ["1,1,1,1,1", "0,37,600,0,5"])
def test_append_is_rotate_then_append(kv, HKV, G, d, page, lens):
    """The same bits as the two calls one after the other, in the pools and in the queries, everywhere."""
    T = tsl()
    lens = [int(x) for x in lens.split(",")]
    starts = [3, 0, 77, 1, 15]
    B, rows = len(lens), sum(lens)
    max_pages = (max(s + n for s, n in zip(starts, lens)) + page - 1) // page
    pages = B * max_pages
    ctx = _context(T, kv, HKV, G, d, page, B, max_pages, pages)
    kind = F32 if kv == "fp32" else BF
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, max_pages).to(DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    extra = 3                                                     # rows behind the last sequence
    k, v, q = _rows(rows + extra, HKV, d, kind, 1), _rows(rows + extra, HKV, d, kind, 2), _rows(rows + extra, HKV * G, d, kind, 3)
    pos = (torch.arange(rows + extra, device=DEV) * 131 % 100000).to(torch.int32)
    for r, pairs, cfg in ((d, False, BANDS), (d // 2, True, PLAIN), (d - 14, False, YARN)):
        rope = ctx.rope(r, interleaved=pairs, **cfg)
        kr = torch.empty(rows + extra, HKV, d, dtype=kind, device=DEV)
        ctx.rotate(rope, k, pos, kr)
        want = [_pool(kv, pages, HKV, page, d) for _ in range(2)]
        ctx.append_prompt(kr, v, cu, table, *want, starts=st)
        for q_kind in (None, BF, F32):
            got = [_pool(kv, pages, HKV, page, d) for _ in range(2)]
            q_out = q_want = None
            if q_kind is not None:
                q_out, q_want = (torch.full((rows + extra, HKV * G, d), 9.0, dtype=q_kind, device=DEV) for _ in range(2))
                ctx.rotate(rope, q, pos, q_want)
            before = T.ts_kernel_count(ctx.handle)
            ctx.append_rotated(rope, k, v, pos, cu, table, *got, starts=st, q=None if q_kind is None else q, q_out=q_out)
            assert T.ts_kernel_count(ctx.handle) == before + 1 and ctx.status() == 0
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            if q_kind is not None:
                assert torch.equal(q_out, q_want)


def test_append_records_what_has_no_place():
    T = tsl()
    B, HKV, d = 3, 8, 128
    ctx = _context(T, "bf16", HKV, 4, d, 16, B, 2, 6)
    rope = ctx.rope()
    k = _rows(9, HKV, d, BF, 1)
    pos = torch.zeros(9, dtype=torch.int32, device=DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(B, 2)
    cases = [([0, 3, 6, 9], [0, -1, 0], table, "TS_ERR_SEQ_LEN", 1), ([0, 3, 6, 9], [0, 30, 0], table, "TS_ERR_SEQ_LEN", None),
             ([0, 3, 2, 9], [0, 0, 0], table, "TS_ERR_SEQ_LEN", None),
             ([0, 3, 6, 9], [0, 0, 0], torch.tensor([[0, 1], [6, 3], [4, 5]], dtype=torch.int32, device=DEV), "TS_ERR_PAGE_OOB", 1)]
    for cu, starts, tab, want, untouched in cases:
        pools = [_pool("bf16", 6, HKV, 16, d) for _ in range(2)]
        ctx.append_rotated(rope, k, k, pos, torch.tensor(cu, dtype=torch.int32, device=DEV), tab, *pools,
                           starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
        assert ctx.status() == T.STATUS_CODE[want]
        assert torch.equal(pools[0][0, :, :3].transpose(0, 1), k[:3])          # (positions 0: as they are)
        if untouched is not None:
            assert torch.all(pools[0][2 * untouched:2 * untouched + 2] == 3.0)


def test_captured_and_replayed_on_another_stream():
    T = tsl()
    B, HKV, d, rows = 2, 8, 128, 40
    ctx = _context(T, "bf16", HKV, 4, d, 16, B, 4, 8)
    rope = ctx.rope(**BANDS)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(B, 4)
    cu = torch.tensor([0, 13, 40], dtype=torch.int32, device=DEV)
    k, v, q = _rows(rows, HKV, d, BF, 1), _rows(rows, HKV, d, BF, 2), _rows(rows, 32, d, BF, 3)
    pos = torch.arange(rows, dtype=torch.int32, device=DEV)
    pools, q_out = [_pool("bf16", 8, HKV, 16, d) for _ in range(2)], torch.zeros(rows, 32, d, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ctx.append_rotated(rope, k, v, pos, cu, table, *pools, q=q, q_out=q_out)
    for seed in (5, 6):
        k.copy_(_rows(rows, HKV, d, BF, seed))
        pos.add_(1000)
        g.replay()
        want, q_want = [_pool("bf16", 8, HKV, 16, d) for _ in range(2)], torch.zeros_like(q_out)
        ctx.append_rotated(rope, k, v, pos, cu, table, *want, q=q, q_out=q_want)
        assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1]) and torch.equal(q_out, q_want)
    assert ctx.status() == 0
