"""ts_prompt_attend where the scores are far from zero, to the ends of fp32.

Queries and keys are small whole numbers times a power of two, so that scores are exact in fp32 and in the oracle.
Their differences are zero or at least 32: a row's weights are 1 / t for its t largest scores and below 2^-40
elsewhere. An output is off by its rounding (2^-8), that of 1 / t and of t terms' sum (t 2^-23), what the others
weigh (2^-40 times the largest value), and the rounding of the weights to bf16 (2^-8 of each): they are taken
against a maximum that is itself rounded, so the t largest need not be 1 before they are divided by their sum.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from parity import tsl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("H,Hkv", [(8, 2), (4, 4)])
@pytest.mark.parametrize("e", [4, 10, 12, 14, 20, 50])
@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("rise", [False, True])
def test_scores_of_any_size(H, Hkv, e, scale, rise):
    T, d, lens = tsl(), 64, [300, 1, 400]
    n = sum(lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(e)
    q, k = (torch.randint(-7, 8, (n, heads, d), generator=g, device=DEV).float() for heads in (H, Hkv))
    if rise:                                   # scores that grow along the prompts, from ones near zero
        k *= torch.exp2(torch.linspace(-e, e, n, device=DEV).round()).view(n, 1, 1)
        q *= 2.0 ** e
        k[:, :, 8:] = 0                        # (few elements, and one size to a key: exact all the same)
    else:
        q, k = q * 2.0 ** e, k * 2.0 ** e
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    v = torch.randn(n, Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    cu = [0, 300, 301, 701]
    out, lse = torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(n, H, device=DEV)
    ctx = T.Context(H, Hkv, d, T.TS_KV_Q4, 3, 1, 1)
    ctx.prompt_attend(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), out, lse, scale=scale)
    assert ctx.status() == 0
    qn, kn, vn, on, ln = (x.double().cpu().numpy() for x in (q, k, v, out, lse))
    for lo, hi in zip(cu[:-1], cu[1:]):
        for r in range(lo, hi, 1 if hi - lo < 3 else 7):
            for h in range(H):
                kk, vv = kn[lo:r + 1, h // (H // Hkv)], vn[lo:r + 1, h // (H // Hkv)]
                s = scale * (kk @ qn[r, h])
                want, wl, w = O.attention(qn[r, h], kk, vv, scale)
                near = s > s.max() - 32
                if np.any(near & (s < s.max())):
                    continue                   # (rising scores begin near zero: ordinary rows, tested elsewhere)
                t = int(near.sum())
                tol = np.abs(want) * 2.0 ** -8 + (w @ np.abs(vv)) * (2.0 ** -8 + t * 2.0 ** -22) + np.abs(vv).max() * 2.0 ** -38 + 1e-30
                assert np.all(np.abs(on[r, h] - want) <= tol), (r, h, t, on[r, h][:3], want[:3])
                assert abs(ln[r, h] - wl) <= abs(wl) * 2.0 ** -22 + 2.0 ** -20


@pytest.mark.parametrize("H,Hkv,d", [(8, 4, 64), (32, 8, 128)])
def test_a_wait_limit_far_below_any_wait_is_reported_and_leaves_the_context_usable(H, Hkv, d):
    # every role gives up at its first wait that is not over at once; copies and products in flight are waited for
    T, n = tsl(), 3000
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    q, k, v = (torch.randn(n, heads, d, generator=g, device=DEV).to(torch.bfloat16) for heads in (H, Hkv, Hkv))
    cu = torch.tensor([0, 700, n], dtype=torch.int32, device=DEV)
    ctx = T.Context(H, Hkv, d, T.TS_KV_Q4, 2, 1, 1)
    ref, out = (torch.zeros(n, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ctx.prompt_attend(q, k, v, cu, ref)
    assert ctx.status() == 0
    T.ts_set_wait_limit(ctx.handle, 1)
    for _ in range(3):
        ctx.prompt_attend(q, k, v, cu, out)
        assert ctx.status() == T.STATUS_CODE["TS_ERR_TIMEOUT"]
    T.ts_set_wait_limit(ctx.handle, 1_000_000_000)
    out.zero_()
    ctx.prompt_attend(q, k, v, cu, out)
    assert ctx.status() == 0 and torch.equal(out, ref)
