"""The Python binding without a GPU: what it imports, and the calls that it refuses before the library is reached."""
import builtins

import pytest
import torch

import token_level_sparse_gb300 as T


class Reached(Exception):
    pass


class OnDevice(torch.Tensor):
    """A tensor that says that it is on device 0, the current one here."""

    def get_device(self):
        return 0


class Elsewhere(OnDevice):
    """One that says that it is on another."""

    def get_device(self):
        return 1


def _on(t):
    return t.as_subclass(OnDevice)


@pytest.fixture
def context(monkeypatch):
    """Makes contexts without the library, which raises Reached where a call gets to it."""
    made = []

    def make(*a, **kw):
        made.append(T.Context(*a, **kw))
        return made[-1]

    def reached(*a):
        raise Reached

    monkeypatch.setattr(T, "ts_create", lambda cfg: 1)
    monkeypatch.setattr(T, "_check", reached)
    monkeypatch.setattr(T, "_current_stream", lambda: 0)
    monkeypatch.setattr(T, "library", reached)
    T._torch()
    monkeypatch.setattr(T, "_device", lambda: 0)
    monkeypatch.setattr(T, "ts_page_bytes", lambda cfg: 2 * 16 * (68 if cfg.kv_dtype == T.TS_KV_Q4 else 512))
    yield make
    for c in made:
        c.handle = None                                            # (there is nothing to destroy)


def test_a_context_needs_no_torch(context, monkeypatch):
    real = builtins.__import__

    def refuse(name, *a, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ImportError(name)
        return real(name, *a, **kw)

    monkeypatch.setattr(builtins, "__import__", refuse)
    with pytest.raises(ImportError):
        import torch as _                                          # noqa: F401
    c = context(8, 2, 128, T.TS_KV_Q4, 2, 4, 8)
    assert c.max_tokens == 64


H, HKV, D, B = 8, 2, 128, 2


def _calls(c):
    """Every call of a 4-bit context that takes tensors, and good ones for it (but for where they are)."""
    f32, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    pool = torch.zeros(8, HKV, 16 * (D // 2 + D // 32), dtype=torch.uint8)
    a = dict(q=torch.zeros(B, H, D), k_pool=pool, v_pool=pool, page_table=torch.zeros(B, 4, dtype=i32),
             seq_lens=torch.ones(B, dtype=i32))
    out = dict(out=torch.zeros(B, H, D), lse=torch.zeros(B, H))
    listed = dict(idx=torch.zeros(B, 9, dtype=i32), count=torch.zeros(B, dtype=i32))
    score = {x: a[x] for x in ("q", "k_pool", "page_table", "seq_lens")} | dict(
        vote=torch.zeros(B, 64), skip=torch.zeros(B, dtype=torch.uint8))
    rows = torch.zeros(5, HKV, D, dtype=bf)
    packed = dict(cu_rows=torch.tensor([0, 2, 5], dtype=i32), page_table=a["page_table"], k_pool=pool, v_pool=pool,
                  starts=torch.zeros(B, dtype=i32))
    prm = T.params()
    return {
        "attend": (c.attend, a | out),
        "score": (c.score, score),
        "score_fn": (lambda **kw: c.score_fn(prm, **kw), score),
        "sparse_attend": (c.sparse_attend, {x: a[x] for x in ("q", "k_pool", "v_pool", "page_table")} | out | listed),
        "decode_step": (lambda **kw: c.decode_step(params=prm, **kw),
                        a | out | listed | dict(vote=torch.zeros(B, 64), hit=torch.zeros(B, dtype=torch.uint8))),
        "append_kv": (c.append_kv, {x: a[x] for x in ("page_table", "seq_lens", "k_pool", "v_pool")}
                      | dict(k_new=torch.zeros(B, HKV, D, dtype=bf), v_new=torch.zeros(B, HKV, D, dtype=bf))),
        "append_prompt": (c.append_prompt, packed | dict(k=rows, v=rows)),
        "read_kv": (c.read_kv, packed | dict(k_out=torch.zeros(5, HKV, D), v_out=torch.zeros(5, HKV, D))),
    }


CALLS = ("attend", "score", "score_fn", "sparse_attend", "decode_step", "append_kv", "append_prompt", "read_kv")


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_shape_or_type_are_refused(context, name):
    c = context(H, HKV, D, T.TS_KV_Q4, B, 4, 8)
    call, good = _calls(c)[name]
    good = {key: _on(t) for key, t in good.items()}
    with pytest.raises(Reached):
        call(**good)
    # buffers for more sequences than the call has, and scores in rows of a wider matrix
    for key in {"seq_lens", "out", "lse", "count", "idx", "vote", "page_table", "hit", "skip", "k_pool"} & set(good):
        if (name, key) != ("append_kv", "seq_lens"):
            with pytest.raises(Reached):
                call(**(good | {key: _on(torch.cat([good[key], good[key][:1]]))}))
    if "q" in good:
        with pytest.raises(Reached):
            call(**(good | {"q": good["q"].flatten(1)}))
        for bad in (good["q"].flatten(1)[:, :-1], good["q"].flatten(), good["q"][:, :1], good["q"].transpose(0, 1)):
            with pytest.raises(T.TokenSelectError):
                call(**(good | {"q": bad}))
    if "vote" in good:
        with pytest.raises(Reached):
            call(**(good | {"vote": _on(torch.zeros(B, 99))[:, :30]}))
    for key, t in good.items():
        smaller = t[:-1] if t.dim() == 1 or key.endswith("pool") or key in ("idx", "vote") else t[..., :-1].contiguous()
        wrong = [smaller, t.to(torch.float64), t.as_subclass(torch.Tensor), t.as_subclass(Elsewhere)]
        if t.dtype == torch.float32 and key != "vote":
            wrong.append(t.to(torch.bfloat16))
        if key in ("k_new", "v_new", "k", "v"):
            wrong += [t.float(), t.to(torch.float16)]              # the type of another pool; as wide, but another type
        if key.endswith("pool"):
            wrong = [smaller, t.as_subclass(torch.Tensor), t.as_subclass(Elsewhere)]         # (a pool is bytes, of any type)
        if key in ("skip", "hit"):
            wrong = [smaller, t.int(), t.as_subclass(torch.Tensor), t.as_subclass(Elsewhere)]
        if (name, key) == ("append_kv", "seq_lens"):
            wrong = wrong[1:]                                      # (fewer lengths are fewer sequences)
        if key == "cu_rows":
            wrong = [t.long(), t.as_subclass(torch.Tensor), t.as_subclass(Elsewhere)]        # (fewer boundaries are fewer sequences)
        if key in ("q", "page_table", "vote", "idx"):
            wrong.append(t.repeat_interleave(2, -1)[..., ::2])     # (not dense)
        for bad in wrong:
            with pytest.raises(T.TokenSelectError) as e:
                call(**(good | {key: bad}))
            assert e.value.status in (T.STATUS_CODE["TS_ERR_SHAPE"], T.STATUS_CODE["TS_ERR_INVALID_ARG"]), (key, bad.dtype)


def test_prompts_on_another_device_are_refused(context):
    c = context(H, HKV, D, T.TS_KV_Q4, B, 4, 8)
    q, k = (_on(torch.zeros(5, heads, D, dtype=torch.bfloat16)) for heads in (H, HKV))
    good = dict(q=q, k=k, v=k, cu_rows=_on(torch.tensor([0, 2, 5], dtype=torch.int32)), out=q, lse=_on(torch.zeros(5, H)))
    with pytest.raises(Reached):
        c.prompt_attend(**good)
    for key, t in good.items():
        for there in (torch.Tensor, Elsewhere):
            with pytest.raises(T.TokenSelectError):
                c.prompt_attend(**(good | {key: t.as_subclass(there)}))


def test_rows_for_a_pool_that_holds_them_as_they_are(context):
    c = context(H, HKV, D, T.TS_KV_F32, B, 4, 8)
    good = dict(k_new=torch.zeros(B, HKV, D), v_new=torch.zeros(B, HKV, D), page_table=torch.zeros(B, 4, dtype=torch.int32),
                seq_lens=torch.ones(B, dtype=torch.int32), k_pool=torch.zeros(1), v_pool=torch.zeros(1))
    good = {key: _on(t) for key, t in good.items()}
    for bad in (torch.zeros(B, HKV, D, dtype=torch.bfloat16), torch.zeros(B, HKV, D - 1), torch.zeros(B - 1, HKV, D)):
        with pytest.raises(T.TokenSelectError):
            c.append_kv(**(good | {"k_new": _on(bad)}))
    for fine in (torch.zeros(B, HKV, D), torch.zeros(B + 1, HKV, D), torch.zeros(B, HKV * D, dtype=torch.int32)):
        with pytest.raises(Reached):
            c.append_kv(**(good | {"k_new": _on(fine)}))
