"""ts_keep_rows on the GPU (bytes that move as they are), and a round of drafted tokens from end to end."""
import math

import numpy as np
import pytest
import torch

from oracle import draft_oracle as D
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
POOLS = [("bf16", 8, 4, 128, 16), ("bf16", 4, 2, 64, 16), ("bf16", 8, 1, 128, 1), ("f32", 8, 4, 128, 16), ("f32", 4, 1, 64, 1),
         ("q4", 3, 2, 128, 16), ("q4", 8, 2, 64, 16), ("q4", 1, 1, 64, 16)]


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _setup(kv, HKV, G, d, page, lens, layers, seed=0):
    T = tsl()
    rng = np.random.default_rng(seed)
    np_ = [(n + page - 1) // page for n in lens]
    pages = sum(np_) + 2
    table = np.full((len(lens), max(np_)), 0, dtype=np.int32)
    perm, at = rng.permutation(pages), 0
    for b, n in enumerate(np_):
        table[b, :n] = perm[at:at + n]
        at += n
    kind = {"bf16": T.TS_KV_BF16, "f32": T.TS_KV_F32, "q4": T.TS_KV_Q4}[kv]
    shape = (pages, HKV, 16 * (d // 2 + d // 32)) if kv == "q4" else (pages, HKV, page, d * (2 if kv == "bf16" else 4))
    pools = [torch.from_numpy(rng.integers(0, 256, (layers, *shape), dtype=np.uint8)).to(DEV) for _ in range(2)]
    ctx = T.Context(HKV * G, HKV, d, kind, len(lens), max(np_), pages, page)
    return T, ctx, table, pools


def _typed(kv, pool):
    return pool if kv == "q4" else pool.view(BF if kv == "bf16" else torch.float32)


def _want(kv, pools, table, page, d, lens, trees, paths):
    """Rows moved one after another, in bytes."""
    out = [p.cpu().numpy().copy() for p in pools]
    for b, (n, t) in enumerate(zip(lens, trees)):
        for j, src in enumerate(paths[b]):
            s, e = n - t + src, n - t + j
            for x in out:
                a, z = x[:, table[b, s // page]], x[:, table[b, e // page]]
                if kv != "q4":
                    z[:, :, e % page] = a[:, :, s % page]
                    continue
                for nb in range(d // 64):
                    for width, base in ((32, nb * 512), (2, d * 8 + nb * 32)):
                        z[:, :, base + e % 16 * width:base + e % 16 * width + width] = \
                            a[:, :, base + s % 16 * width:base + s % 16 * width + width]
    return out


@pytest.mark.parametrize("kv,HKV,G,d,page", POOLS)
@pytest.mark.parametrize("layers", [1, 3])
def test_rows_move_as_they_are(kv, HKV, G, d, page, layers):
    lens, trees = [1, 40, 300, 77, 64, 500, 30], [1, 17, 64, 5, 64, 400, 0]
    rng = np.random.default_rng(1)
    paths = [[0], [0, 1, 5, 16], sorted(rng.choice(64, 20, replace=False).tolist()), [], list(range(64)),
             sorted(rng.choice(400, 290, replace=False).tolist()), []]
    T, ctx, table, pools = _setup(kv, HKV, G, d, page, lens, layers)
    most = max(len(p) for p in paths)
    path = _i32([p + [-1] * (most - len(p)) for p in paths])
    want = _want(kv, pools, table, page, d, lens, trees, paths)
    new = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    arg = [_typed(kv, p if layers > 1 else p[0]) for p in pools]
    cu = _i32(np.concatenate([[0], np.cumsum(trees)]))
    ctx.keep_rows(path, _i32([len(p) for p in paths]), cu, _i32(lens), _i32(table), *arg, new_lens=new)
    assert ctx.status() == 0
    for a, b in zip(pools, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert new.tolist() == [n - t + len(p) for n, t, p in zip(lens, trees, paths)]


def test_errors_leave_the_sequence():
    T, ctx, table, pools = _setup("bf16", 8, 4, 128, 16, [60, 60], 1)
    before = [p.clone() for p in pools]
    arg = [_typed("bf16", p[0]) for p in pools]
    bad = [([0, 2, 2], 3, "TS_ERR_INVALID_ARG"), ([0, 3, 1], 3, "TS_ERR_INVALID_ARG"), ([0, 1, 9], 3, "TS_ERR_INVALID_ARG"),
           ([-1, 1, 2], 3, "TS_ERR_INVALID_ARG"), ([0, 1, 2], 4, "TS_ERR_CAPACITY"), ([0, 1, 2], -1, "TS_ERR_INVALID_ARG")]
    for row, n, status in bad:
        new = torch.full((2,), 7, dtype=torch.int32, device=DEV)
        ctx.keep_rows(_i32([row, [0, 1, 2]]), _i32([n, 2]), _i32([0, 9, 18]), _i32([60, 60]), _i32(table), *arg, new_lens=new)
        assert ctx.status() == T.STATUS_CODE[status] and new.tolist() == [60, 53]
        assert all(torch.equal(a, b) for a, b in zip(pools, before))
    for cu, lens in (([0, 9, 18], [5, 60]), ([0, 9, 3], [60, 60]), ([0, 9, 18], [60, 10 ** 6]), ([4, 9, 18], [60, 60])):
        ctx.keep_rows(_i32([[0, 1, 2]] * 2), _i32([3, 3]), _i32(cu), _i32(lens), _i32(table), *arg)
        assert ctx.status() == T.STATUS_CODE["TS_ERR_SEQ_LEN"]
        assert all(torch.equal(a, b) for a, b in zip(pools, before))
    ctx.keep_rows(_i32([[0, 1, 2]] * 2), _i32([3, 3]), _i32([0, 9, 18]), _i32([60, 60]), _i32(table), *arg, total=10)
    assert ctx.status() == T.STATUS_CODE["TS_ERR_SEQ_LEN"]
    # a page outside the pool: its rows stay, the others move
    t = table.copy()
    t[0, 3] = 10 ** 6
    ctx.keep_rows(_i32([[0, 8, -1], [0, 1, -1]]), _i32([2, 2]), _i32([0, 16, 32]), _i32([60, 60]), _i32(t), *arg)
    assert ctx.status() == T.STATUS_CODE["TS_ERR_PAGE_OOB"] and all(torch.equal(a, b) for a, b in zip(pools, before))
    lens = _i32([60, 60])
    with pytest.raises(T.TokenSelectError):
        ctx.keep_rows(_i32([[0], [0]]), _i32([1, 1]), _i32([0, 9, 18]), lens, _i32(table), *arg, new_lens=lens)


@pytest.mark.parametrize("HKV,G,d", [(8, 4, 128), (4, 2, 64)])
def test_rounds_of_drafts_from_end_to_end(HKV, G, d):
    """Three rounds, captured once as a graph and replayed: drafts appended with their positions, attended to as a tree,
    verified, kept. The cache then holds what appending the kept tokens one by one gives, bit for bit, and the outputs of
    every round are those of the definition over it."""
    T = tsl()
    B, layers, most, V, max_pages = 3, 2, 12, 50, 8
    pages, H = B * max_pages, HKV * G
    ctx = T.Context(H, HKV, d, T.TS_KV_BF16, B, max_pages, pages)
    rope = ctx.rope(d // 2, base=500000.0, scaling="bands", factor=8.0, original=64, low=1.0, high=4.0)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rng = np.random.default_rng(3)
    table = _i32(rng.permutation(pages).reshape(B, max_pages))
    pools = [torch.zeros(layers, pages, HKV, 16, d, dtype=BF, device=DEV) for _ in range(2)]
    plain = [torch.zeros(layers, pages, HKV, 16, d, dtype=BF, device=DEV) for _ in range(2)]
    lens = [20, 1, 45]                                            # certain tokens, the root not among them
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    cu0 = _i32(np.concatenate([[0], np.cumsum(lens)]))
    pos0 = _i32(np.concatenate([np.arange(n) for n in lens]))
    for layer in range(layers):
        k, v = randn(sum(lens), HKV, d), randn(sum(lens), HKV, d)
        for p in (pools, plain):
            ctx.append_rotated(rope, k, v, pos0, cu0, table, p[0][layer], p[1][layer])
    trees = [most, 5, 9]
    par = [[-1] + [int(rng.integers(0, i)) for i in range(1, t)] for t in trees]
    depth = [[0] * t for t in trees]
    bits = []
    for b, t in enumerate(trees):
        anc = []
        for i in range(t):
            p = par[b][i]
            depth[b][i] = depth[b][p] + 1 if i else 0
            anc.append((anc[p] if i else 0) | 1 << i)
        bits.append(anc)
    rows = sum(trees)
    cu, parents = _i32(np.concatenate([[0], np.cumsum(trees)])), _i32([x for p in par for x in p])
    mask = _i32([[x] for anc in bits for x in anc])
    seq_b = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(trees, device=DEV))
    deep = _i32([x for t in depth for x in t])
    # static buffers of the graph
    certain = _i32(lens)
    q, k, v = randn(layers, rows, H, d), randn(layers, rows, HKV, d), randn(layers, rows, HKV, d)
    q_rot, out = torch.zeros(layers, rows, H, d, dtype=BF, device=DEV), torch.zeros(layers, rows, H, d, dtype=BF, device=DEV)
    lse = torch.zeros(layers, rows, H, device=DEV)
    tokens, target, draft = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(rows, V, device=DEV), torch.zeros(rows, V, device=DEV)
    u, un = torch.zeros(rows, device=DEV), torch.zeros(B, device=DEV)
    path, count, nxt = torch.zeros(B, most, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    size = _i32(trees)

    def step():
        pos = (certain[seq_b] + deep).to(torch.int32)
        total = (certain + size).to(torch.int32)
        for layer in range(layers):
            ctx.append_rotated(rope, k[layer], v[layer], pos, cu, table, pools[0][layer], pools[1][layer], starts=certain,
                               q=q[layer], q_out=q_rot[layer])
            ctx.tree_attend(q_rot[layer], pools[0][layer], pools[1][layer], table, total, cu, mask, out[layer], lse[layer])
        ctx.verify_tree(tokens, parents, cu, target, draft, u, un, path, count, nxt)
        ctx.keep_rows(path, count, cu, total, table, *pools, new_lens=certain)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    scale, long_paths = 1 / math.sqrt(d), 0
    for rnd in range(3):
        for t in (q, k, v):
            t.copy_(randn(*t.shape))
        z = torch.randn(rows, V, generator=g, device=DEV)
        target.copy_(torch.softmax(z, 1))
        draft.copy_(torch.softmax(z + 0.3 * torch.randn(rows, V, generator=g, device=DEV), 1))
        tok = [int(rng.integers(V)) for _ in range(rows)]
        dn = draft.double().cpu().numpy()
        for b, t in enumerate(trees):
            lo = int(cu[b])
            for i in range(1, t):
                tok[lo + i] = int(rng.choice(V, p=dn[lo + par[b][i]] / dn[lo + par[b][i]].sum()))
        tokens.copy_(_i32(tok))
        u.copy_(torch.rand(rows, generator=g, device=DEV))
        un.copy_(torch.rand(B, generator=g, device=DEV))
        graph.replay()
        assert ctx.status() == 0
        new = list(lens)
        for b, t in enumerate(trees):
            lo, hi = int(cu[b]), int(cu[b + 1])
            want, token = D.verify(tok[lo:hi], par[b], target[lo:hi].cpu().numpy(), draft[lo:hi].cpu().numpy(), u[lo:hi].cpu().numpy(),
                                   float(un[b]), False)
            assert path[b].tolist() == want + [-1] * (most - len(want)) and int(count[b]) == len(want) and int(nxt[b]) == token
            long_paths += len(want) > 1
            # the definition over the plain cache and the drafts' own rows
            for layer in range(layers):
                n = lens[b]
                pos = torch.arange(n, device=DEV)
                page = table[b].long()[pos // 16]
                f, a = rope.read()
                posd = [n + x for x in depth[b]]
                kd = D.rotate(k[layer, lo:hi].double().cpu().numpy(), posd, f, a, d // 2, False)
                kd = torch.from_numpy(kd).to(BF).double().numpy()             # (the cache's rounding)
                kk = np.concatenate([plain[0][layer][page, :, pos % 16].double().cpu().numpy(), kd])
                vv = np.concatenate([plain[1][layer][page, :, pos % 16].double().cpu().numpy(), v[layer, lo:hi].double().cpu().numpy()])
                for i in range(t):
                    seen = D.tree_seen(n + t, t, i, bits[b][i])
                    for h in (0, H - 1):
                        qq = q_rot[layer, lo + i, h].double().cpu().numpy()
                        o, wl, w = D.tree_attend(qq, kk[:, h // G], vv[:, h // G], seen, scale)
                        # one bf16 step of a key element that rounds the other way moves a score by 2^-8 |q k| at most: 2^-8 covers it
                        # beside the weights' and the outputs' own 2^-8 each
                        el = scale * float(np.max(np.abs(kk[:, h // G]) @ np.abs(qq))) * (d + 16) * 2.0 ** -24
                        step1 = scale * float(np.max(np.abs(kk[:, h // G]) * np.abs(qq))) * 2.0 ** -7
                        tol = (w @ np.abs(vv[:, h // G])) * (2.0 ** -8 + 2 * (el + step1) + 2.0 ** -16) + np.abs(o) * 2.0 ** -8
                        assert np.all(np.abs(out[layer, lo + i, h].double().cpu().numpy() - o) <= tol)
                        assert abs(float(lse[layer, lo + i, h]) - wl) <= el + step1 + 2.0 ** -16
            new[b] += len(want)
            # the kept rows, appended behind one another with the positions that they have there
            one = _i32([0, len(want)])
            keep = torch.tensor([lo + i for i in want], device=DEV)
            at = _i32([lens[b]])
            pos = _i32([lens[b] + depth[b][i] for i in want])
            assert pos.tolist() == list(range(lens[b], lens[b] + len(want)))
            for layer in range(layers):
                sub = table[b:b + 1].contiguous()
                ctx.append_rotated(rope, k[layer, keep].contiguous(), v[layer, keep].contiguous(), pos, one, sub,
                                   plain[0][layer], plain[1][layer], starts=at)
        assert certain.tolist() == new
        lens = new
        for b in range(B):
            pos = torch.arange(lens[b], device=DEV)
            page = table[b].long()[pos // 16]
            for a, z2 in zip(pools, plain):
                assert torch.equal(a[:, page, :, pos % 16], z2[:, page, :, pos % 16])
    assert long_paths > 0
