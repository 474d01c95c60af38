"""What is measured of decoding with drafted tokens: inputs, plain forms and calls.

Five operators, the steps of one round of drafted tokens over a paged cache:

* ``rotate``  rotary positions of query or key rows (``Context.rotate``);
* ``append``  new K rows, rotated on the way, and V rows into the paged cache, with the queries of the
              same rows rotated beside them (``Context.append_rotated``);
* ``tree``    attention of a tree of drafted tokens over the whole cache (``Context.tree_attend``);
* ``verify``  which drafted tokens the target keeps, and the token behind them, from given random
              numbers (``Context.verify_tree``);
* ``keep``    the kept tokens' K and V rows moved to the front of the draft's (``Context.keep_rows``).

Rows are packed: sequence b has rows cu[b] .. cu[b + 1] - 1. Pools are [num_pages][H_kv][16][d]. Row 0
of a sequence's tree is its root (the last token that is certain), a parent comes before its children.

Where ``own`` is false ``run`` computes in plain torch operations and needs no library.
"""
import math

import torch

own = False

P = 16                      # tokens per page
DEV = "cuda"

# head geometries of the library's pools: (KV heads, query heads per KV head, d)
GEO_BF16 = [(8, 4, 128), (4, 7, 128), (8, 1, 128), (4, 2, 64), (2, 8, 128)]
GEO_F32 = [(4, 1, 64), (2, 4, 64), (8, 4, 128)]


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the queries of a decode batch, one token each, made ready for the decode step (bf16 in, fp32 out)
        dict(name="rotate_token", op="rotate", H=32, d=128, starts="1000,17,131072,4096,65535,2,300,30001",
             lens="1,1,1,1,1,1,1,1", rot=128, layout="half", scaling="plain", src="bf16", dst="fp32"),
        # the queries of three prompts, cut from a fused projection, with frequencies scaled by bands
        dict(name="rotate_prompt", op="rotate", H=32, d=128, starts="0,5000,120000", lens="20000,777,12345", rot=128,
             layout="half", scaling="bands", src="bf16", dst="bf16"),
        # a model whose pairs are neighbours and which turns half of each head
        dict(name="rotate_part", op="rotate", H=8, d=64, starts="3,200000", lens="4001,9000", rot=32, layout="pairs",
             scaling="linear", src="fp32", dst="fp32"),
        # the current token of a decode batch: K rotated and appended, V appended, Q rotated
        dict(name="append_token", op="append", H=32, HKV=8, d=128, starts="999,16,131071,4095,65534,1,299,30000",
             lens="1,1,1,1,1,1,1,1", rot=128, layout="half", scaling="bands", kv="bf16", q="fp32"),
        # the rows of three prompts behind what their sequences hold already
        dict(name="append_prompt", op="append", H=32, HKV=8, d=128, starts="0,5000,7", lens="20000,777,12345", rot=128,
             layout="half", scaling="yarn", kv="bf16", q="bf16"),
        # a small tree for four short chats: the latency of a single small call
        dict(name="tree_short", op="tree", HKV=8, G=4, d=128, lens="37,333,4096,1777", trees="8,8,8,8", kind="tree"),
        # a draft of 64 tokens over one 128K sequence
        dict(name="tree_128k", op="tree", HKV=8, G=4, d=128, lens="131057", trees="64", kind="tree"),
        # trees of a batch of eight sequences of 32K to 250K tokens, one of them without a draft
        dict(name="tree_batch", op="tree", HKV=4, G=7, d=128, lens="32801,45000,60013,80000,101111,139000,190001,249999",
             trees="16,5,33,1,26,0,18,24", kind="tree"),
        # a chain for one sequence of a small vocabulary: the latency of the walk
        dict(name="verify_chain", op="verify", trees="6", V=32001, draw="chain", draft="probs"),
        # trees of a serving batch over a large vocabulary, siblings drawn without replacement
        dict(name="verify_batch", op="verify", trees=",".join(str(17 + (i * 29) % 48) for i in range(32)), V=128256,
             draw="distinct", draft="probs"),
        # one layer, one sequence
        dict(name="keep_one", op="keep", HKV=8, d=128, lens="4100", trees="16", layers=1, kv="bf16"),
        # all layers of a batch in one call
        dict(name="keep_layers", op="keep", HKV=8, d=128, lens=",".join(str(70 + (i * 37) % 300) for i in range(16)),
             trees=",".join(str(16 + (i * 13) % 49) for i in range(16)), layers=32, kv="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _join(v):
    return ",".join(map(str, v))


def draw(rng):
    op = rng.choice(["rotate", "append", "tree", "tree", "verify", "keep"])
    if op in ("rotate", "append"):
        B = _log(rng, 1, 24)
        lens = [_log(rng, 1, 30000 // B) for _ in range(B)]
        case = dict(op=op, lens=_join(lens), layout=rng.choice(["half", "pairs"]),
                    scaling=rng.choice(["plain", "linear", "base", "bands", "yarn"]))
        if op == "rotate":
            d = rng.choice([64, 128])
            return dict(case, H=rng.choice([1, 4, 8, 24, 28, 32]), d=d, starts=_join(_log(rng, 1, 1000000) for _ in range(B)),
                        rot=rng.choice([d, d // 2, 2 * rng.randint(2, d // 2)]), src=rng.choice(["bf16", "fp32"]),
                        dst=rng.choice(["bf16", "fp32"]))
        kv = rng.choice(["bf16", "bf16", "fp32"])
        HKV, G, d = rng.choice(GEO_BF16 if kv == "bf16" else GEO_F32)
        return dict(case, H=HKV * G, HKV=HKV, d=d, starts=_join(_log(rng, 1, 60000 // B) for _ in range(B)),
                    rot=rng.choice([d, d // 2, 2 * rng.randint(2, d // 2)]), kv=kv, q=rng.choice(["none", "bf16", "fp32"]))
    if op == "tree":
        HKV, G, d = rng.choice(GEO_BF16)
        B = _log(rng, 1, 24)
        trees = [rng.choice([0, 1, 2, _log(rng, 1, 64), _log(rng, 1, max(1, 400 // B))]) for _ in range(B)]
        trees[0] = max(1, trees[0])
        lens = [max(t, _log(rng, 1, 400000 // B)) for t in trees]
        return dict(op=op, HKV=HKV, G=G, d=d, lens=_join(lens), trees=_join(trees), kind=rng.choice(["tree", "tree", "chain"]))
    if op == "verify":
        B = _log(rng, 1, 32)
        return dict(op=op, trees=_join(_log(rng, 1, 64) for _ in range(B)), V=_log(rng, 2, 128256),
                    draw=rng.choice(["chain", "same", "distinct"]), draft=rng.choice(["probs", "probs", "none"]))
    kv = rng.choice(["bf16", "fp32"])
    HKV, _, d = rng.choice(GEO_BF16 if kv == "bf16" else GEO_F32)
    B = _log(rng, 1, 16)
    trees = [_log(rng, 1, 64) for _ in range(B)]
    return dict(op=op, HKV=HKV, d=d, lens=_join(t + rng.randint(0, 200) for t in trees), trees=_join(trees),
                layers=_log(rng, 1, 32), kv=kv)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _keeps(trees):
    """Tokens that a kept path has: the root and a few drafts."""
    return [min(t, 1 + (3 * b + 2) % 5) for b, t in enumerate(trees)]


def work(case):
    """Inputs once, outputs once."""
    op = case["op"]
    if op == "rotate":
        rows, es = sum(_ints(case["lens"])), {"bf16": 2, "fp32": 4}
        n = rows * case["H"]
        return {"bytes": n * case["d"] * (es[case["src"]] + es[case["dst"]]) + rows * 4, "flops": n * case["rot"] * 3}
    if op == "append":
        rows, es = sum(_ints(case["lens"])), {"bf16": 2, "fp32": 4, "none": 0}
        kv, q = rows * case["HKV"] * case["d"], rows * case["H"] * case["d"]
        qb = q * (es[case["kv"]] + es[case["q"]]) if case["q"] != "none" else 0
        return {"bytes": kv * 4 * es[case["kv"]] + qb + rows * 4,
                "flops": rows * case["rot"] * 3 * (case["HKV"] + (case["H"] if qb else 0))}
    if op == "tree":
        n, t, H, d = _ints(case["lens"]), _ints(case["trees"]), case["HKV"] * case["G"], case["d"]
        toks = sum(x for x, y in zip(n, t) if y)
        return {"bytes": toks * case["HKV"] * d * 4 + sum(t) * H * (4 * d + 4), "flops": 4 * d * H * sum(x * y for x, y in zip(n, t))}
    if op == "verify":
        # the row that the token behind the path is drawn from, the nodes and the random numbers
        t = _ints(case["trees"])
        rows = 2 if case["draft"] == "probs" else 1
        return {"bytes": len(t) * rows * case["V"] * 4 + sum(t) * 16, "flops": len(t) * case["V"] * 4}
    # every kept row but the root is read and written
    moved = sum(k - 1 for k in _keeps(_ints(case["trees"])))
    es = 2 if case["kv"] == "bf16" else 4
    return {"bytes": max(1, moved) * case["layers"] * case["HKV"] * case["d"] * es * 4, "flops": 0}


# ----------------------------------------------------------------- inputs

class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV)

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device=DEV)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device=DEV)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return _int32(out)


_TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
BASE, FACTOR, ORIGINAL = 500000.0, 8.0, 8192


def _rope_args(case):
    """What a model's configuration says of its positions."""
    args = dict(rot_dim=case["rot"], base=BASE, interleaved=case["layout"] == "pairs", scaling=case["scaling"])
    if case["scaling"] != "plain":
        args["factor"] = FACTOR
    if case["scaling"] == "bands":
        args.update(original=ORIGINAL, low=1.0, high=4.0)
    if case["scaling"] == "yarn":
        args.update(original=ORIGINAL, low=1.0, high=32.0)
    return args


def _table(lens, g):
    """A page table over a pool whose pages are scattered; its pages."""
    np_ = [(x + P - 1) // P for x in lens]
    perm = g.perm(max(1, sum(np_))).to(torch.int32)
    table = torch.zeros(len(lens), max(1, max(np_)), dtype=torch.int32, device=DEV)
    at = 0
    for b, x in enumerate(np_):
        table[b, :x] = perm[at:at + x]
        at += x
    return table, perm.shape[0]


def _parents(trees, kind, rng):
    """Parents of every tree's nodes by levels: 1, then 4, 6, 8, ... nodes; or a chain."""
    out = []
    for t in trees:
        par, level, size = [-1] if t else [], [0], 4
        while len(par) < t:
            if kind == "chain":
                par.append(len(par) - 1)
                continue
            nodes = range(len(par), min(t, len(par) + size))
            par += sorted(level[int(u * len(level))] for u in rng[len(par):len(par) + len(nodes)])
            level, size = list(nodes), size + 2
        out.append(par)
    return out


def _mask(parents, words):
    """int32 [rows][words]: bit j of a row is set where node j is the row's own or an ancestor of it."""
    rows = []
    for par in parents:
        anc = []
        for i, p in enumerate(par):
            anc.append((anc[p] if p >= 0 else 0) | (1 << i))
        rows += anc
    low = [[(x >> (32 * w)) & 0xffffffff for w in range(words)] for x in rows] or [[0] * words]
    return _int32([[v - (1 << 32) if v >> 31 else v for v in r] for r in low])


def _context(kv, H, HKV, d, max_batch, max_pages, num_pages):
    import token_level_sparse_gb300 as T
    return T.Context(H, HKV, d, {"bf16": T.TS_KV_BF16, "fp32": T.TS_KV_F32, "4bit": T.TS_KV_Q4}[kv], max_batch, max_pages, num_pages)


def prepare(case, seed):
    op, g = case["op"], _Gen(seed)
    st = {"case": case}
    if op in ("rotate", "append"):
        lens, starts = _ints(case["lens"]), _ints(case["starts"])
        rows, H, d = sum(lens), case["H"], case["d"]
        b = torch.repeat_interleave(torch.arange(len(lens), device=DEV), torch.tensor(lens, device=DEV))
        cu = _cu(lens)
        st["positions"] = (torch.arange(rows, device=DEV) - cu.long()[b] + torch.tensor(starts, device=DEV)[b]).to(torch.int32)
        if op == "rotate":
            # column range of a projection
            st["x"] = g.normal(rows, (H + 2) * d).to(_TYPE[case["src"]])[:, :H * d].view(rows, H, d)
            st["out"] = torch.zeros(rows, H, d, dtype=_TYPE[case["dst"]], device=DEV)
            if own:
                st["ctx"] = _context("4bit", H, H, d, 1, 1, 1)
        else:
            HKV = case["HKV"]
            qkv = g.normal(rows, (H + 2 * HKV) * d).to(_TYPE[case["kv"]])
            st["q"] = qkv[:, :H * d].view(rows, H, d)
            st["k"] = qkv[:, H * d:(H + HKV) * d].view(rows, HKV, d)
            st["v"] = qkv[:, (H + HKV) * d:].view(rows, HKV, d)
            st["table"], pages = _table([s + n for s, n in zip(starts, lens)], g)
            st["cu"], st["starts"] = cu, _int32(starts)
            st["k_pool"], st["v_pool"] = (torch.zeros(pages, HKV, P, d, dtype=_TYPE[case["kv"]], device=DEV) for _ in range(2))
            st["q_out"] = torch.zeros(rows, H, d, dtype=_TYPE[case["q"]], device=DEV) if case["q"] != "none" else None
            if own:
                st["ctx"] = _context(case["kv"], H, HKV, d, len(lens), st["table"].shape[1], pages)
        if own:
            st["rope"] = st["ctx"].rope(**_rope_args(case))
        return st
    if op == "verify":
        trees, V = _ints(case["trees"]), case["V"]
        B, T = len(trees), max(trees)
        parents = _parents(trees, "chain" if case["draw"] == "chain" else "tree", g.uniform(T + 64).tolist())
        rows = sum(trees)
        # both distributions of a node lie near one another, as a good drafter's do
        st["target"], st["draft"] = torch.empty(rows, V, device=DEV), torch.empty(rows, V, device=DEV)
        for r0 in range(0, rows, 64):
            n = min(64, rows - r0)
            z = 2.5 * g.normal(n, V)
            st["target"][r0:r0 + n] = torch.softmax(z, dim=1)
            st["draft"][r0:r0 + n] = torch.softmax(z + 0.8 * g.normal(n, V), dim=1)
        cu = _cu(trees)
        st["cu"], st["trees"] = cu, trees
        st["parents"] = _int32([p for par in parents for p in par])
        # every node's token from its parent's draft distribution, siblings distinct where the case says so
        first = cu.long()[:-1]
        tokens = torch.zeros(rows, dtype=torch.int64, device=DEV)
        for i in range(1, T):
            live = [k for k in range(B) if trees[k] > i]
            at = torch.tensor(live, device=DEV)
            par = torch.tensor([parents[k][i] for k in live], device=DEV)
            w = st["draft"][first[at] + par].clone()
            if case["draw"] == "distinct" or case["draft"] == "none":
                for k, b in enumerate(live):
                    sib = [j for j in range(1, i) if parents[b][j] == parents[b][i]]
                    if sib:
                        w[k, tokens[first[b] + torch.tensor(sib, device=DEV)]] = 0
            c = torch.cumsum(w.double(), dim=1)
            u = g.uniform(len(live)).double()[:, None] * c[:, -1:]
            tokens[first[at] + i] = torch.searchsorted(c, u, right=True)[:, 0].clamp(max=V - 1)
        st["tokens"] = tokens.to(torch.int32)
        st["u"], st["u_next"] = g.uniform(rows), g.uniform(B)
        if case["draft"] == "none":
            st["draft"] = None
        st["path"] = torch.zeros(B, T, dtype=torch.int32, device=DEV)
        st["count"], st["next"] = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
        if own:
            st["ctx"] = _context("4bit", 8, 8, 64, B, 1, 1)
        return st
    lens, trees, d = _ints(case["lens"]), _ints(case["trees"]), case["d"]
    HKV, B = case["HKV"], len(lens)
    st["table"], pages = _table(lens, g)
    st["cu"], st["seq_lens"], st["lens"], st["trees"] = _cu(trees), _int32(lens), lens, trees
    if op == "tree":
        H = HKV * case["G"]
        st["q"] = (1.5 * g.normal(sum(trees), H, d)).to(torch.bfloat16)
        st["k_pool"], st["v_pool"] = (torch.empty(pages, HKV, P, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        for pool in (st["k_pool"], st["v_pool"]):
            for p0 in range(0, pages, 4096):
                pool[p0:p0 + 4096] = g.normal(min(4096, pages - p0), HKV, P, d)
        parents = _parents(trees, case["kind"], g.uniform(max(trees) + 128).tolist())
        st["mask"] = _mask(parents, (max(trees) + 31) // 32)
        st["out"] = torch.zeros(sum(trees), H, d, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.zeros(sum(trees), H, device=DEV)
        if own:
            st["ctx"] = _context("bf16", H, HKV, d, B, st["table"].shape[1], pages)
        return st
    st["k_pool"], st["v_pool"] = (torch.empty(case["layers"], pages, HKV, P, d, dtype=_TYPE[case["kv"]], device=DEV) for _ in range(2))
    for pool in (st["k_pool"], st["v_pool"]):
        for layer in range(case["layers"]):
            pool[layer] = g.normal(pages, HKV, P, d)
    # the root and a few drafts, ascending
    keeps = _keeps(trees)
    st["path"] = torch.zeros(B, max(keeps), dtype=torch.int32, device=DEV)
    for b, (t, k) in enumerate(zip(trees, keeps)):
        if k > 1:
            st["path"][b, 1:k] = (g.perm(t - 1)[:k - 1].sort().values + 1).to(torch.int32)
    st["count"], st["new_lens"] = _int32(keeps), torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        G = 4 if (HKV, d) == (8, 128) else {(4, 128): 7, (4, 64): 2, (2, 128): 8, (2, 64): 4}[HKV, d]
        if case["kv"] == "fp32" and (HKV, d) == (4, 64):
            G = 1
        st["ctx"] = _context(case["kv"], HKV * G, HKV, d, B, st["table"].shape[1], pages)
    return st


# ------------------------------------------------------------ plain forms

def _frequencies(case):
    """Radians per position of every pair, and the factor of what is turned (64 bits)."""
    r, kind = case["rot"], case["scaling"]
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    base = BASE * FACTOR ** (r / (r - 2)) if kind == "base" and r > 2 else BASE
    f = torch.pow(torch.tensor(base, dtype=torch.float64, device=DEV), -2 * i / r)
    if kind == "linear":
        return f / FACTOR, 1.0
    if kind == "bands":
        t = ((ORIGINAL * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - t) * f / FACTOR + t * f, 1.0
    if kind == "yarn":
        at = [r * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(BASE)) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return t * f / FACTOR + (1 - t) * f, 0.1 * math.log(FACTOR) + 1
    return f, 1.0


def _turn(x, positions, case):
    """Rows turned by their positions, in 32 bits; the angles in 64."""
    f, a = _frequencies(case)
    ang = positions.double()[:, None] * f
    cos, sin = (a * torch.cos(ang)).float()[:, None], (a * torch.sin(ang)).float()[:, None]
    r = case["rot"]
    y = x.float()
    if case["layout"] == "pairs":
        x1, x2 = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
    else:
        x1, x2 = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
    return torch.cat([turned, y[..., r:]], dim=-1)


def _plain_rotate(st):
    st["out"].copy_(_turn(st["x"], st["positions"], st["case"]))
    return st["out"]


def _place(st, n_rows):
    """Page and slot of every packed row."""
    cu = st["cu"].long()
    row = torch.arange(n_rows, device=DEV)
    b = torch.searchsorted(cu[1:], row, right=True)
    pos = row - cu[b] + st["starts"].long()[b]
    return st["table"].long()[b, pos // P], pos % P


def _plain_append(st):
    page, slot = _place(st, st["k"].shape[0])
    st["k_pool"][page, :, slot] = _turn(st["k"], st["positions"], st["case"]).to(st["k_pool"].dtype)
    st["v_pool"][page, :, slot] = st["v"]
    if st["q_out"] is not None:
        st["q_out"].copy_(_turn(st["q"], st["positions"], st["case"]))
        return st["k_pool"], st["v_pool"], st["q_out"]
    return st["k_pool"], st["v_pool"]


def _plain_tree(st):
    case = st["case"]
    HKV, G, d = case["HKV"], case["G"], case["d"]
    at = 0
    for b, (n, t) in enumerate(zip(st["lens"], st["trees"])):       # (each its own length)
        if t == 0:
            continue
        page = st["table"][b, :(n + P - 1) // P].long()
        k, v = (st[x][page].permute(1, 0, 2, 3).reshape(HKV, -1, d)[:, :n].float() for x in ("k_pool", "v_pool"))
        q = st["q"][at:at + t].float().view(t, HKV, G, d).permute(1, 0, 2, 3).reshape(HKV, t * G, d)
        s = torch.matmul(q, k.transpose(1, 2)).view(HKV, t, G, n) / math.sqrt(d)
        j = torch.arange(t, device=DEV)
        seen = (st["mask"][at:at + t][:, j // 32] >> (j % 32)) & 1
        s[..., n - t:].masked_fill_((seen == 0)[None, :, None, :], -math.inf)
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        o = torch.matmul((e / z).view(HKV, t * G, n), v).view(HKV, t, G, d)
        st["out"][at:at + t] = o.permute(1, 0, 2, 3).reshape(t, HKV * G, d).to(torch.bfloat16)
        st["lse"][at:at + t] = (m + torch.log(z))[..., 0].permute(1, 0, 2).reshape(t, HKV * G)
        at += t
    return st["out"], st["lse"]


def _plain_verify(st):
    """All sequences side by side, node after node (a child comes behind its parent)."""
    case, B, V = st["case"], len(st["trees"]), st["case"]["V"]
    first = st["cu"].long()[:-1]
    size = st["cu"].long()[1:] - first
    one = torch.ones(B, dtype=torch.float64, device=DEV)
    cur, c, Z, W = torch.zeros(B, dtype=torch.int64, device=DEV), 0 * one, one, one
    gone = torch.zeros(B, V, dtype=torch.bool, device=DEV)              # tokens refused at this node (draft "none")
    seq = torch.arange(B, device=DEV)
    path = torch.zeros_like(st["path"])
    count = torch.ones_like(cur)
    for i in range(1, max(st["trees"])):
        live = size > i
        node = torch.where(live, first + i, first)
        mine = live & (st["parents"].long()[node] == cur)
        x, u = st["tokens"].long()[node], st["u"][node].double()
        p = st["target"][first + cur].double()
        if st["draft"] is not None:
            q = st["draft"][first + cur].double()
            px, qx = p[seq, x], q[seq, x]
            yes = mine & (u * qx * Z < (px - c * qx).clamp(min=0) * W)
            no = mine & ~yes
            c = torch.where(no, c + torch.where(W > 0, Z / W, 0 * W), c)
            Z = torch.where(no, (p - c[:, None] * q).clamp(min=0).sum(1), Z)
            if case["draw"] == "distinct":
                W = torch.where(no, W - qx, W)
        else:
            px = torch.where(gone[seq, x], 0 * one, p[seq, x])
            yes = mine & (u * Z < px)
            no = mine & ~yes
            Z = torch.where(no, Z - px, Z)
            gone[seq, x] |= no
            gone &= ~yes[:, None]
        c, Z, W = (torch.where(yes, v, w) for v, w in ((0 * one, c), (one, Z), (one, W)))
        path[seq, torch.where(yes, count, 0)] = torch.where(yes, i, path[seq, 0].long()).to(torch.int32)
        cur = torch.where(yes, i, cur)
        count = count + yes
    p = st["target"][first + cur].double()
    r = (p - c[:, None] * st["draft"][first + cur].double()).clamp(min=0) if st["draft"] is not None else p * ~gone
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    cum = torch.cumsum(r, dim=1)
    token = torch.searchsorted(cum, st["u_next"].double()[:, None] * cum[:, -1:], right=True)[:, 0].clamp(max=V - 1)
    behind = torch.arange(path.shape[1], device=DEV)[None, :] >= count[:, None]
    st["path"].copy_(path.masked_fill(behind, -1))
    st["count"].copy_(count)
    st["next"].copy_(token)
    return st["path"], st["count"], st["next"]


def _plain_keep(st):
    first = (st["seq_lens"] - (st["cu"][1:] - st["cu"][:-1])).long()
    k = torch.arange(st["path"].shape[1], device=DEV)
    b, k = (k[None, :] < st["count"][:, None]).nonzero(as_tuple=True)
    src, dst = first[b] + st["path"].long()[b, k], first[b] + k
    table = st["table"].long()
    for pool in (st["k_pool"], st["v_pool"]):
        pool[:, table[b, dst // P], :, dst % P] = pool[:, table[b, src // P], :, src % P]
    st["new_lens"].copy_(first + st["count"])
    return st["k_pool"], st["v_pool"], st["new_lens"]


_PLAIN = {"rotate": _plain_rotate, "append": _plain_append, "tree": _plain_tree, "verify": _plain_verify, "keep": _plain_keep}


def run(st):
    if not own:
        return _PLAIN[st["case"]["op"]](st)
    op, ctx = st["case"]["op"], st["ctx"]
    if op == "rotate":
        ctx.rotate(st["rope"], st["x"], st["positions"], st["out"])
        return st["out"]
    if op == "append":
        ctx.append_rotated(st["rope"], st["k"], st["v"], st["positions"], st["cu"], st["table"], st["k_pool"], st["v_pool"],
                           starts=st["starts"], q=None if st["q_out"] is None else st["q"], q_out=st["q_out"])
        return (st["k_pool"], st["v_pool"]) if st["q_out"] is None else (st["k_pool"], st["v_pool"], st["q_out"])
    if op == "tree":
        ctx.tree_attend(st["q"], st["k_pool"], st["v_pool"], st["table"], st["seq_lens"], st["cu"], st["mask"], st["out"], st["lse"])
        return st["out"], st["lse"]
    if op == "verify":
        ctx.verify_tree(st["tokens"], st["parents"], st["cu"], st["target"], st["draft"], st["u"], st["u_next"], st["path"],
                        st["count"], st["next"], distinct=st["case"]["draw"] == "distinct")
        return st["path"], st["count"], st["next"]
    ctx.keep_rows(st["path"], st["count"], st["cu"], st["seq_lens"], st["table"], st["k_pool"], st["v_pool"], st["new_lens"])
    return st["k_pool"], st["v_pool"], st["new_lens"]


# ------------------------------------------------------------------ exact

def _exact_turn(x, positions, case):
    """Each pair as a complex number times a e^(i pos f), pair by pair."""
    r, kind, y = case["rot"], case["scaling"], x.double().clone()
    for i in range(r // 2):
        base = BASE * FACTOR ** (r / (r - 2)) if kind == "base" and r > 2 else BASE
        f, a = math.exp(-2 * i / r * math.log(base)), 1.0
        if kind == "linear":
            f /= FACTOR
        elif kind == "bands":
            wave = 2 * math.pi / f
            if wave > ORIGINAL / 1.0:
                f /= FACTOR
            elif wave >= ORIGINAL / 4.0:
                t = (ORIGINAL / wave - 1.0) / (4.0 - 1.0)
                f = (1 - t) * f / FACTOR + t * f
        elif kind == "yarn":
            index = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
            lo, hi = max(0, math.floor(index(32.0))), min(r - 1, math.ceil(index(1.0)))
            t = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f, a = f / FACTOR * t + f * (1 - t), 1 + 0.1 * math.log(FACTOR)
        e1, e2 = (2 * i, 2 * i + 1) if case["layout"] == "pairs" else (i, i + r // 2)
        z = torch.complex(x[..., e1].double(), x[..., e2].double())
        w = torch.polar(torch.full(positions.shape, a, dtype=torch.float64, device=DEV), positions.double() * f)
        z = z * w[:, None]
        y[..., e1], y[..., e2] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    if case["op"] == "verify":
        return None                                       # whole numbers only
    if case["op"] == "tree" and work(case)["flops"] > 2.5e11:
        return None
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "rotate":
        return _exact_turn(st["x"], st["positions"], case)
    if case["op"] == "append":
        pools = [torch.zeros(st["k_pool"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
        k, at = _exact_turn(st["k"], st["positions"], case), 0
        for b, (s, n) in enumerate(zip(_ints(case["starts"]), _ints(case["lens"]))):
            pos = torch.arange(s, s + n, device=DEV)
            page = st["table"][b].long()[torch.div(pos, P, rounding_mode="floor")]
            pools[0][page, :, pos % P] = k[at:at + n]
            pools[1][page, :, pos % P] = st["v"][at:at + n].double()
            at += n
        return tuple(pools) if st["q_out"] is None else (*pools, _exact_turn(st["q"], st["positions"], case))
    if case["op"] == "tree":
        HKV, G, d = case["HKV"], case["G"], case["d"]
        out = torch.zeros(sum(st["trees"]), HKV * G, d, dtype=torch.float64, device=DEV)
        lse = torch.zeros(sum(st["trees"]), HKV * G, dtype=torch.float64, device=DEV)
        at, mask = 0, st["mask"].cpu().tolist()
        for b, (n, t) in enumerate(zip(st["lens"], st["trees"])):
            hide = torch.zeros(t, n, dtype=torch.bool, device=DEV)
            for i in range(t):
                hide[i, n - t:] = torch.tensor([not (mask[at + i][j // 32] >> (j % 32)) & 1 for j in range(t)], device=DEV)
            for g in range(HKV if t else 0):
                rows = st["table"][b, :(n + P - 1) // P].long()
                k, v = (st[x][rows, g].reshape(-1, d)[:n].double() for x in ("k_pool", "v_pool"))
                for h in range(g * G, (g + 1) * G):
                    x = torch.einsum("id,jd->ij", st["q"][at:at + t, h].double(), k) / math.sqrt(d)
                    x[hide] = -math.inf
                    z = torch.logsumexp(x, dim=1)
                    out[at:at + t, h], lse[at:at + t, h] = torch.exp(x - z[:, None]) @ v, z
            at += t
        return out, lse
    pools = [st[x].double() for x in ("k_pool", "v_pool")]
    for b, (n, t, k) in enumerate(zip(st["lens"], st["trees"], _keeps(st["trees"]))):
        path = st["path"][b].tolist()
        for x in pools:
            for i in range(k):                            # ascending: a row is read before it is written over
                s, e = n - t + path[i], n - t + i
                x[:, int(st["table"][b, e // P]), :, e % P] = x[:, int(st["table"][b, s // P]), :, s % P].clone()
    return (*pools, None)
