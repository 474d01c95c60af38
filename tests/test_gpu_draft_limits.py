"""Calls for drafted tokens at their limits: offsets past 32 bits, refused arguments, short wait limits, and their
neighbours among the library's calls."""
import ctypes
import math

import numpy as np
import pytest
import torch

from parity import tsl
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=I32).to(DEV)


def test_pages_past_four_gigabytes():
    """The same sequence in the first pages of a small pool and in the last of a large one: the same bits."""
    T = tsl()
    HKV, G, d, n, t, big = 8, 4, 128, 300, 20, 140000
    assert big * HKV * 16 * d > 1 << 31
    got = []
    for pages in (64, big):
        ctx = T.Context(HKV * G, HKV, d, T.TS_KV_BF16, 1, 20, pages)
        rope = ctx.rope()
        g = torch.Generator(device=DEV)
        g.manual_seed(1)
        pools = [torch.empty(pages, HKV, 16, d, dtype=BF, device=DEV) for _ in range(2)]
        last = torch.arange(pages - 20, pages, device=DEV)
        for p in pools:
            p[last] = 0
        table = last.to(I32).view(1, 20)
        k, v = (torch.randn(n, HKV, d, generator=g, device=DEV).to(BF) for _ in range(2))
        q, out = torch.randn(t, HKV * G, d, generator=g, device=DEV).to(BF), torch.zeros(t, HKV * G, d, dtype=BF, device=DEV)
        pos = torch.arange(n, dtype=I32, device=DEV)
        ctx.append_rotated(rope, k, v, pos, _i32([0, n]), table, *pools)
        ctx.tree_attend(q, *pools, table, _i32([n]), _i32([0, t]), None, out)
        first = [p[last].clone() for p in pools]
        ctx.keep_rows(_i32([[0, 3, 7, 19]]), _i32([4]), _i32([0, t]), _i32([n]), table, *pools)
        assert ctx.status() == 0
        got.append([out] + first + [p[last].clone() for p in pools])
        del pools
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_rows_past_four_gigabytes():
    T = tsl()
    rows, heads, d, step = 2600, 4, 128, 1 << 20
    ctx = T.Context(heads, heads, d, T.TS_KV_Q4, 1, 1, 1)
    rope = ctx.rope()
    wide = torch.empty(rows * step, dtype=BF, device=DEV)
    x = wide.as_strided((rows, heads, d), (step, d, 1))
    x.copy_(torch.randn(rows, heads, d, device=DEV))
    pos, want, dense = torch.arange(rows, dtype=I32, device=DEV), torch.empty(rows, heads, d, dtype=BF, device=DEV), x.contiguous()
    ctx.rotate(rope, dense, pos, want)
    out = torch.empty(rows, heads, d, dtype=BF, device=DEV)
    ctx.rotate(rope, x, pos, out)
    ctx.rotate(rope, x, pos, x)
    assert torch.equal(out, want) and torch.equal(x, want)
    del wide, x
    # the second sequence's distributions begin past 2^32 bytes
    V, n0, n1 = 1 << 20, 1024, 5
    vc = T.Context(4, 4, 64, T.TS_KV_Q4, 2, 1, 1)
    target = torch.zeros(n0 + n1, V, device=DEV)
    assert n0 * V * 4 >= 1 << 32
    for i in range(n1):
        target[n0 + i, 1000 * (i + 1)] = 1.0
    tokens = torch.zeros(n0 + n1, dtype=I32, device=DEV)
    tokens[n0 + 1:] = _i32([1000, 2000, 3000, 7])
    parents = _i32([-1] + [0] * (n0 - 1) + [-1, 0, 1, 2, 3])
    path, count, nxt = (torch.zeros(s, dtype=I32, device=DEV) for s in ((2, 6), (2,), (2,)))
    vc.verify_tree(tokens, parents, _i32([0, n0, n0 + n1]), target, None, torch.full((n0 + n1,), 0.5, device=DEV),
                   torch.zeros(2, device=DEV), path, count, nxt)
    assert vc.status() == 0 and count.tolist() == [1, 4] and path[1].tolist() == [0, 1, 2, 3, -1, -1] and nxt.tolist() == [-1, 4000]


def test_a_single_token_is_what_the_sparse_attention_gives():
    """One draft per sequence over the whole cache, beside ts_sparse_attend over a list of every token (fp32 outputs)."""
    c = Case(8, 4, 128, lens=[700, 33, 1], trees=[1, 1, 1], mask=None, seed=3)
    c.k_pool.nan_to_num_(0.0)
    c.v_pool.nan_to_num_(0.0)
    c.run()
    idx, out, lse = torch.zeros(3, 700, dtype=I32, device=DEV), torch.zeros(3, 32, 128, device=DEV), torch.zeros(3, 32, device=DEV)
    for b, n in enumerate(c.lens):
        idx[b, :n] = torch.arange(n, device=DEV)
    table = c.table.copy()
    table[table < 0] = 0
    c.ctx.sparse_attend(c.q.float().contiguous(), c.k_pool, c.v_pool, c.dev(table), idx, c.dev(c.lens), out, lse)
    # weights and outputs rounded to bf16: 2^-8 each of what is at most the largest value
    assert float((out - c.out.float()).abs().max()) <= 2 * 2.0 ** -8 * float(max(v.abs().max() for v in c.v))
    assert float((lse - c.lse).abs().max()) <= 2.0 ** -14


def test_short_wait_limits_leave_a_usable_context():
    """Every wait gives up at once; the call after it, with the limit back, is right."""
    T = tsl()
    c = Case(8, 4, 128, lens=[5000, 300, 64], trees=[60, 33, 5], seed=4)
    c.run()
    want, wl = c.out.clone(), c.lse.clone()
    for _ in range(3):
        T.ts_set_wait_limit(c.ctx.handle, 1)
        c.run()
        assert c.ctx.status() in (0, T.STATUS_CODE["TS_ERR_TIMEOUT"])
        T.ts_set_wait_limit(c.ctx.handle, 1000000000)
        c.out.fill_(0)
        c.run()
        assert c.ctx.status() == 0 and torch.equal(c.out, want) and torch.equal(c.lse, wl)


def test_rows_behind_the_last_sequence_and_padded_batches():
    """A buffer of more rows than the trees take, and sequences of no drafts at either end."""
    c = Case(4, 2, 64, lens=[0, 50, 9, 70, 20], trees=[0, 7, 0, 3, 0], extra=500, seed=5)
    c.run().check()
    assert torch.all(c.out[10:] == 7.0) and torch.all(c.lse[10:] == 7.0)
    c = Case(4, 2, 64, lens=[40, 50], trees=[0, 0], extra=6, seed=6)
    c.run()
    assert c.ctx.status() == 0 and torch.all(c.out == 7.0)


def test_two_graphs_of_one_context():
    """Their parts share the context's room: replayed one behind the other, each gives its own outputs."""
    a = Case(8, 4, 128, lens=[9000], trees=[40], seed=7)
    b = Case(8, 4, 128, lens=[9000], trees=[25], seed=8)
    b.ctx = a.ctx
    a.run()
    b.run()
    want = (a.out.clone(), b.out.clone())
    graphs, s = [], torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for c in (a, b):
        args = (c.q, c.k_pool, c.v_pool, c.dev(c.table), c.dev(c.lens), c.dev(c.cu), c.mask_tensor(), c.out, c.lse)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.ctx.tree_attend(*args)
        graphs.append((g, args))
    for _ in range(2):
        a.out.fill_(0)
        b.out.fill_(0)
        for g, _ in graphs + graphs[::-1]:
            g.replay()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    assert a.ctx.status() == 0


def test_refused_arguments():
    """The library's own checks, past the binding's: nothing runs, nothing is written."""
    T = tsl()
    ctx = T.Context(32, 8, 128, T.TS_KV_BF16, 2, 4, 8)
    rope, wide = ctx.rope(), T.Rope(128)
    small = T.Context(4, 4, 64, T.TS_KV_Q4, 2, 4, 8)
    h, buf = ctx.handle, torch.zeros(1 << 20, dtype=BF, device=DEV)
    p, ints = buf.data_ptr(), torch.zeros(4096, dtype=I32, device=DEV)
    i = ints.data_ptr()
    f = torch.zeros(4096, device=DEV).data_ptr()
    SHAPE, INVALID = T.STATUS_CODE["TS_ERR_SHAPE"], T.STATUS_CODE["TS_ERR_INVALID_ARG"]
    lib = T.library()

    def call(fn, good, status, **bad):
        args = dict(good)
        args.update(bad)
        before = T.ts_kernel_count(args["ctx"])
        assert getattr(lib, fn)(*args.values()) == status, (fn, bad)
        assert T.ts_kernel_count(args["ctx"]) == before

    r = rope.handle
    rotate = dict(ctx=h, rope=r, x=p, xs=128 * 4, dtype=1, heads=4, pos=i, total=3, out=p + 65536, os=128 * 4, odtype=1, stream=None)
    for bad in (dict(rope=None), dict(x=None), dict(pos=None), dict(out=None), dict(dtype=2), dict(odtype=5), dict(x=p + 2), dict(xs=516),
                dict(out=p, odtype=0), dict(out=p, os=128 * 8)):
        call("ts_rotate", rotate, INVALID, **bad)
    for bad in (dict(xs=128), dict(os=504), dict(heads=0), dict(total=-1), dict(xs=1 << 32), dict(ctx=small.handle, rope=wide.handle)):
        call("ts_rotate", rotate, SHAPE, **bad)
    append = dict(ctx=h, rope=r, k=p, ks=1024, v=p, vs=1024, pos=i, cu=i, starts=None, B=2, total=3, table=i, kp=p, vp=p, q=p, qs=4096,
                  qo=p + 65536, qos=4096, qod=1, stream=None)
    for bad in (dict(k=None), dict(pos=None), dict(cu=None), dict(table=None), dict(q=None), dict(qo=None), dict(k=p + 8), dict(ks=1028),
                dict(qod=2), dict(qo=p, qod=0), dict(qo=p, qos=8192), dict(qo=p + 4)):
        call("ts_append_rotated", append, INVALID, **bad)
    for bad in (dict(B=0), dict(B=3), dict(total=-1), dict(ks=1016), dict(qs=4088), dict(qos=4088)):
        call("ts_append_rotated", append, SHAPE, **bad)
    tree = dict(ctx=h, q=p, qs=4096, kp=p, vp=p, table=i, lens=i, cu=i, mask=i, words=1, B=2, total=3, scale=0.0, out=p, os=4096, lse=None,
                stream=None)
    for bad in (dict(q=None), dict(kp=None), dict(lens=None), dict(cu=None), dict(out=None), dict(q=p + 8), dict(qs=4100), dict(scale=math.nan)):
        call("ts_tree_attend", tree, INVALID, **bad)
    for bad in (dict(words=0), dict(words=33), dict(B=3), dict(total=(1 << 24) + 1), dict(qs=4088), dict(os=8)):
        call("ts_tree_attend", tree, SHAPE, **bad)
    verify = dict(ctx=h, tok=i, par=i, cu=i, B=2, total=3, V=30, t=f, ts=30, d=f, ds=30, u=f, un=f, distinct=0, path=i, most=4, count=i,
                  nxt=i, stream=None)
    for bad in (dict(tok=None), dict(par=None), dict(cu=None), dict(t=None), dict(u=None), dict(un=None), dict(path=None), dict(count=None),
                dict(nxt=None)):
        call("ts_verify_tree", verify, INVALID, **bad)
    for bad in (dict(V=0), dict(V=(1 << 20) + 1, ts=1 << 21, ds=1 << 21), dict(ts=29), dict(ds=29), dict(most=0), dict(B=3), dict(total=-1)):
        call("ts_verify_tree", verify, SHAPE, **bad)
    keep = dict(ctx=h, path=i, most=4, count=i + 64, cu=i + 128, lens=i + 256, B=2, total=3, table=i, kp=p, vp=p, layers=2,
                step=ctypes.c_int64(8 * 32768), new=i + 512, stream=None)
    for bad in (dict(path=None), dict(count=None), dict(lens=None), dict(table=None), dict(kp=p + 2), dict(new=i + 256), dict(new=i + 68),
                dict(new=i + 136), dict(new=i + 28), dict(step=ctypes.c_int64(8 * 32768 + 8))):
        call("ts_keep_rows", keep, INVALID, **bad)
    for bad in (dict(layers=0), dict(layers=65536), dict(step=ctypes.c_int64(8 * 32768 - 16)), dict(most=0), dict(B=3), dict(total=-1)):
        call("ts_keep_rows", keep, SHAPE, **bad)
    torch.cuda.synchronize()
    assert ctx.status() == 0 and not bool(ints.any()) and not bool(buf.any())
