"""The binding's calls for drafted tokens without a GPU: what is refused before the library is reached."""
import pytest
import torch

import token_level_sparse_gb300 as T
from test_binding_cpu import Elsewhere, Reached, _on, context  # noqa: F401

H, HKV, D, B, ROWS = 8, 2, 128, 2, 5
I32, F32, BF = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def page_bytes(context, monkeypatch):  # noqa: F811
    monkeypatch.setattr(T, "ts_page_bytes", lambda cfg: 2 * 16 * D * (2 if cfg.kv_dtype == T.TS_KV_BF16 else 4))


class FakeRope:
    handle = 1


def _calls(c):
    rope = FakeRope()
    cu, table = torch.tensor([0, 2, ROWS], dtype=I32), torch.zeros(B, 4, dtype=I32)
    pool = torch.zeros(8, HKV, 16, D, dtype=BF)
    lens, pos = torch.full((B,), 9, dtype=I32), torch.zeros(ROWS, dtype=I32)
    q, k = torch.zeros(ROWS, H, D, dtype=BF), torch.zeros(ROWS, HKV, D, dtype=BF)
    probs = torch.zeros(ROWS, 30)
    paged = dict(page_table=table, k_pool=pool, v_pool=pool, cu_rows=cu)
    return {
        "rotate": (lambda **kw: c.rotate(rope, **kw), dict(x=q, positions=pos, out=torch.zeros(ROWS, H, D))),
        "append_rotated": (lambda **kw: c.append_rotated(rope, **kw),
                           paged | dict(k=k, v=k, positions=pos, starts=torch.zeros(B, dtype=I32), q=q, q_out=torch.zeros(ROWS, H, D))),
        "tree_attend": (c.tree_attend, paged | dict(q=q, seq_lens=lens, mask=torch.zeros(ROWS, 1, dtype=I32), out=q, lse=torch.zeros(ROWS, H))),
        "verify_tree": (c.verify_tree, dict(tokens=pos, parents=pos, cu_rows=cu, target=probs, draft=probs, u=torch.zeros(ROWS),
                                            u_next=torch.zeros(B), path=torch.zeros(B, 3, dtype=I32), count=lens, next_token=lens)),
        "keep_rows": (c.keep_rows, paged | dict(path=torch.zeros(B, 3, dtype=I32), count=lens, seq_lens=lens, new_lens=lens)),
    }


@pytest.mark.parametrize("name", ["rotate", "append_rotated", "tree_attend", "verify_tree", "keep_rows"])
def test_tensors_of_another_shape_or_type_are_refused(context, name):  # noqa: F811
    c = context(H, HKV, D, T.TS_KV_BF16, B, 4, 8)
    call, good = _calls(c)[name]
    good = {key: _on(t) for key, t in good.items()}
    with pytest.raises(Reached):
        call(**good)
    for key in {"starts", "mask", "lse", "draft", "new_lens"} & set(good):
        with pytest.raises(Reached):
            call(**(good | {key: None}))
    for key, t in good.items():
        pool = key.endswith("pool")
        wrong = [t.as_subclass(torch.Tensor), t.as_subclass(Elsewhere)]
        if not pool:
            wrong += [t.to(torch.float64), t.to(torch.float16) if t.is_floating_point() else t.long()]
        if key != "cu_rows":                                       # (fewer boundaries are fewer sequences)
            wrong.append(t[:-1])
        if t.dim() > 1 and not pool and key not in ("path", "mask"):
            wrong.append(t[..., :-1].contiguous())
        if t.dim() > 1 and not pool:
            wrong.append(t.repeat_interleave(2, -1)[..., ::2])     # (not dense)
        if t.dim() == 3:
            wrong += [t[:, :-1].contiguous(), t.flatten(1)]
        for bad in wrong:
            with pytest.raises(T.TokenSelectError) as e:
                call(**(good | {key: bad}))
            assert e.value.status in (T.STATUS_CODE["TS_ERR_SHAPE"], T.STATUS_CODE["TS_ERR_INVALID_ARG"]), (key, bad.dtype, bad.shape)


def test_rows_of_a_wider_matrix_are_taken(context):  # noqa: F811
    c = context(H, HKV, D, T.TS_KV_BF16, B, 4, 8)
    wide = _on(torch.zeros(ROWS, (H + 2 * HKV) * D, dtype=BF))
    q, k = wide[:, :H * D].view(ROWS, H, D), wide[:, H * D:(H + HKV) * D].view(ROWS, HKV, D)
    for name, more in (("rotate", dict(x=q)), ("append_rotated", dict(k=k, q=q)), ("tree_attend", dict(q=q, out=q)),
                       ("verify_tree", dict(target=_on(torch.zeros(ROWS, 40))[:, :30]))):
        call, good = _calls(c)[name]
        with pytest.raises(Reached):
            call(**({key: _on(t) for key, t in good.items()} | more))


def test_types_go_with_the_pool(context):  # noqa: F811
    c = context(H, HKV, D, T.TS_KV_F32, B, 4, 8)
    call, good = _calls(c)["append_rotated"]
    good = {key: _on(t) for key, t in good.items()}
    with pytest.raises(T.TokenSelectError):
        call(**good)                                               # bf16 rows into an fp32 pool
    f32 = good | {key: _on(good[key].float()) for key in ("k", "v", "q", "k_pool", "v_pool")}
    with pytest.raises(Reached):
        call(**f32)
    for bad in (dict(q=None), dict(q_out=None), dict(q=good["q"])):
        with pytest.raises(T.TokenSelectError):
            call(**(f32 | bad))


def test_pools_of_several_layers(context):  # noqa: F811
    c = context(H, HKV, D, T.TS_KV_BF16, B, 4, 8)
    call, good = _calls(c)["keep_rows"]
    good = {key: _on(t) for key, t in good.items()}
    layers = _on(torch.zeros(3, 8, HKV, 16, D, dtype=BF))
    with pytest.raises(Reached):
        call(**(good | dict(k_pool=layers, v_pool=layers)))
    for bad in (layers[:2], layers[:, :7].contiguous(), layers.float(), layers.transpose(0, 1), layers[0]):
        with pytest.raises(T.TokenSelectError):
            call(**(good | dict(k_pool=layers, v_pool=bad)))
    with pytest.raises(T.TokenSelectError):
        call(**(good | dict(k_pool=_on(torch.zeros(3, 7, HKV, 16, D, dtype=BF)), v_pool=_on(torch.zeros(3, 7, HKV, 16, D, dtype=BF)))))
