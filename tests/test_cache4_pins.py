"""CPU pins of the 4-bit cache's oracle and of the new entry points' refusals (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O


def test_round_bf16_agrees_with_torch():
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(5000) * 10.0 ** rng.integers(-38, 38, 5000), [0.0, 1.00390625, 1.01171875, 3.4e38]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).double().numpy()
    assert np.array_equal(O.round_bf16(x), want)


def test_quantise_by_hand():
    x = np.zeros(64)
    x[:6] = [7.0, -7.0, 0.5, 1.5, -2.5, 3.2]              # scale 1: ties to even
    codes, scale = O.q4_quantise(x)
    assert scale.tolist() == [1.0]
    assert codes[0, :6].tolist() == [15, 1, 8, 10, 6, 11] and set(codes[0, 6:]) == {8}
    assert O.q4_values(codes, scale)[:6].tolist() == [7, -7, 0, 2, -2, 3]


def test_quantise_takes_the_nearest_code_and_stays_within_half_a_scale():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((40, 128)) * 10.0 ** rng.integers(-3, 4, (40, 1))).to(torch.bfloat16).double().numpy()
    codes, scale = O.q4_quantise(x)
    v = O.q4_values(codes, scale)
    per = np.repeat(scale, 64, axis=1)
    inside = np.abs(x) <= 7 * per
    assert np.all(np.abs(x - v)[inside] <= per[inside] / 2 * (1 + 1e-12))
    assert np.all(np.abs(v)[~inside] == 7 * per[~inside])
    for u in range(1, 16):
        assert np.all(np.abs(x - v) <= np.abs(x - (u - 8) * per) * (1 + 1e-12))


def test_quantise_of_zeros_and_non_finite_groups():
    x = np.zeros((3, 64))
    x[1, 5], x[1, 6] = np.nan, 2.0
    x[2, 0] = np.inf
    codes, scale = O.q4_quantise(x)
    v = O.q4_values(codes, scale)
    assert np.all(v[0] == 0) and np.all(np.isnan(v[1])) and np.all(np.isnan(v[2]))


@pytest.mark.parametrize("d", [64, 128])
def test_pack_and_pool_values_agree(d):
    rng = np.random.default_rng(d)
    rows = rng.standard_normal((2, 3, 16, d))
    codes, scale = O.q4_quantise(rows)
    pool = np.stack([np.stack([O.q4_pack(codes[p, h], scale[p, h]) for h in range(3)]) for p in range(2)])
    assert pool.shape == (2, 3, 16 * (d // 2 + d // 32))
    assert np.array_equal(O.q4_pool_values(pool, d), O.q4_values(codes, scale))


@pytest.mark.parametrize("G,d", [(1, 64), (4, 64), (7, 128)])
def test_prompt_attention_is_torch_causal_attention(G, d):
    g = torch.Generator().manual_seed(G)
    lens, hkv = [5, 0, 1, 33], 2
    cu = np.concatenate([[0], np.cumsum(lens)])
    q = torch.randn(39, hkv * G, d, generator=g, dtype=torch.float64)
    k, v = (torch.randn(39, hkv, d, generator=g, dtype=torch.float64) for _ in range(2))
    out, lse = O.prompt_attention(q.numpy(), k.numpy(), v.numpy(), cu, 1 / math.sqrt(d))
    for lo, hi in zip(cu[:-1], cu[1:]):
        if lo == hi:
            continue
        want = torch.nn.functional.scaled_dot_product_attention(
            q[lo:hi].transpose(0, 1), k[lo:hi].repeat_interleave(G, 1).transpose(0, 1),
            v[lo:hi].repeat_interleave(G, 1).transpose(0, 1), is_causal=True).transpose(0, 1)
        assert np.allclose(out[lo:hi], want.numpy(), atol=1e-12)
        s = torch.einsum("ihd,jhd->hij", q[lo:hi], k[lo:hi].repeat_interleave(G, 1)) / math.sqrt(d)
        s = s.masked_fill(torch.ones(hi - lo, hi - lo).triu(1).bool(), -math.inf)
        assert np.allclose(lse[lo:hi], torch.logsumexp(s, -1).T.numpy(), atol=1e-12)


@pytest.fixture(scope="module")
def lib():
    from token_level_sparse_gb300 import build
    build.build()
    import token_level_sparse_gb300 as T
    return T.library()


def test_page_bytes(lib):
    import token_level_sparse_gb300 as T
    for kind, per_row in ((T.TS_KV_F32, 512), (T.TS_KV_BF16, 256), (T.TS_KV_Q4, 68)):
        assert T.ts_page_bytes(T.Config(32, 8, 128, 16, kind, 1, 1, 1)) == 8 * 16 * per_row
    assert T.ts_page_bytes(T.Config(8, 4, 64, 16, T.TS_KV_Q4, 1, 1, 1)) == 4 * 16 * 34
    assert T.ts_page_bytes(T.Config(8, 4, 64, 16, 9, 1, 1, 1)) == 0
    assert lib.ts_page_bytes(None) == 0


@pytest.mark.parametrize("cfg,want", [
    ((32, 8, 128, 1), "TS_ERR_UNSUPPORTED"),     # one-token pages
    ((32, 8, 96, 16), "TS_ERR_UNSUPPORTED"),     # head dim
    ((34, 2, 128, 16), "TS_ERR_UNSUPPORTED"),    # 17 query heads per KV head
    ((32, 5, 128, 16), "TS_ERR_INVALID_ARG"),
    ((65, 65, 64, 16), "TS_ERR_UNSUPPORTED"),    # more KV heads than counters
])
def test_four_bit_contexts_refused(lib, cfg, want):
    import token_level_sparse_gb300 as T
    h = ctypes.c_void_p()
    c = T.Config(cfg[0], cfg[1], cfg[2], cfg[3], T.TS_KV_Q4, 1, 10, 10)
    assert lib.ts_create(ctypes.byref(h), ctypes.byref(c)) == T.STATUS_CODE[want]


def test_null_arguments_are_refused(lib):
    import token_level_sparse_gb300 as T
    INVALID = T.STATUS_CODE["TS_ERR_INVALID_ARG"]
    assert lib.ts_attend(None, None, None, None, None, None, 1, 0.0, None, None, None) == INVALID
    assert lib.ts_prompt_attend(None, None, 0, None, 0, None, 0, None, 1, 1, 0.0, None, 0, None, None) == INVALID
    assert lib.ts_append_prompt(None, None, 0, None, 0, None, None, 1, 1, None, None, None, None) == INVALID
    assert lib.ts_read_kv(None, None, None, 1, 1, None, None, None, None, None, None) == INVALID
    assert lib.ts_sparse_attend_noalloc(32, 8, 128, T.TS_KV_Q4, 16, 16, 16, 1, 16, 1, 16, 1, 16, 1, 0.0, 16, None,
                                        None, None) == T.STATUS_CODE["TS_ERR_UNSUPPORTED"]


def test_packed_rows_must_be_dense_inside():
    import token_level_sparse_gb300 as T
    x = torch.zeros(5, 4, 64)
    stride = lambda t: T._row_stride(t, t.shape[0], t.shape[1:])
    assert stride(x) == 256 and stride(x[:, :2]) == 256 and stride(x[:1].expand(1, 4, 64)) == 256
    for bad in (x[:, ::2], x[:, :, ::2], x.transpose(0, 1)):
        with pytest.raises(T.TokenSelectError):
            stride(bad)
