"""Plain fp64 CPU oracle of the 4-bit cache and of the prompt attention (test infrastructure only).

Written from the definitions in include/tokenselect.h, with no code of the CUDA library:

* a group of 64 elements of a row has scale bf16(max|x| / 7) and codes 8 + round(x / scale), ties to
  even, kept in [1, 15]; a code u stands for (u - 8) * scale; a scale of zero gives zeros, a group
  with a NaN or an infinity reads back as NaN;
* the block of a (page, KV head) is codes [d/64][16][32 bytes] (byte j: element 2j low, 2j + 1
  high), then scales bf16 [d/64][16];
* row i of a prompt attends to rows 0 .. i of its own prompt.
"""
from __future__ import annotations

import numpy as np

GROUP = 64
PAGE = 16


def round_bf16(x) -> np.ndarray:
    """fp64 -> the nearest bf16 value (ties to even), as fp64; NaN and infinities stay."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    ok = np.isfinite(x) & (x != 0)
    e = np.maximum(np.frexp(np.where(ok, x, 1.0))[1] - 1, -126)     # exponent; subnormals share the last one
    step = np.ldexp(1.0, e - 7)
    out[ok] = (np.round(x / step) * step)[ok]
    return np.where(np.abs(out) >= np.ldexp(1.0, 128), np.sign(out) * np.inf, out)


def q4_quantise(x):
    """x [..., d] -> codes int [..., d/64, 64] and scales fp64 (bf16 values) [..., d/64]."""
    x = np.asarray(x, dtype=np.float64)
    grp = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(invalid="ignore", over="ignore"):
        scale = round_bf16(np.max(np.abs(grp), axis=-1) / 7.0)
        scale = np.where(np.isnan(grp).any(axis=-1), np.nan, scale)
        live = np.isfinite(scale) & (scale > 0)
        c = np.round(grp / np.where(live, scale, 1.0)[..., None])
    c = np.where(live[..., None], np.clip(c, -7, 7), 0.0)
    return (c + 8).astype(np.int64), scale


def q4_values(codes, scales) -> np.ndarray:
    """The values that codes [..., d/64, 64] and scales [..., d/64] stand for, [..., d]."""
    with np.errstate(invalid="ignore"):
        v = (np.asarray(codes) - 8.0) * np.asarray(scales)[..., None]
    return v.reshape(*v.shape[:-2], -1)


def q4_pack(codes, scales) -> np.ndarray:
    """Codes [16, d/64, 64] and scales [16, d/64] of one (page, KV head) -> its block, uint8."""
    nb = codes.shape[1]
    out = []
    for n in range(nb):
        for t in range(PAGE):
            for j in range(32):
                out.append(int(codes[t, n, 2 * j]) | (int(codes[t, n, 2 * j + 1]) << 4))
    bits = np.asarray(scales, dtype=np.float32).view(np.uint32) >> 16
    for n in range(nb):
        for t in range(PAGE):
            out += [int(bits[t, n]) & 255, int(bits[t, n]) >> 8]
    return np.array(out, dtype=np.uint8)


def q4_pool_values(pool: np.ndarray, d: int) -> np.ndarray:
    """A pool uint8 [num_pages][H_kv][16 (d/2 + d/32)] as values [num_pages][H_kv][16][d]."""
    pages, heads, _ = pool.shape
    nb = d // GROUP
    by = pool[:, :, :PAGE * d // 2].reshape(pages, heads, nb, PAGE, 32)
    codes = np.empty((pages, heads, nb, PAGE, 64), dtype=np.float64)
    codes[..., 0::2] = by & 15
    codes[..., 1::2] = by >> 4
    raw = np.ascontiguousarray(pool[:, :, PAGE * d // 2:]).view(np.uint16).astype(np.uint32) << 16
    scale = raw.view(np.float32).astype(np.float64).reshape(pages, heads, nb, PAGE)
    with np.errstate(invalid="ignore"):
        v = (codes - 8) * scale[..., None]
    return v.transpose(0, 1, 3, 2, 4).reshape(pages, heads, PAGE, d)


def attention(q, k, v, scale):
    """One query q [d] over rows k, v [n, d]: (out [d], lse, weights [n])."""
    s = scale * (k @ q)
    m = np.max(s)
    e = np.exp(s - m)
    z = np.sum(e)
    return (e / z) @ v, m + np.log(z), e / z


def prompt_attention(q, k, v, cu, scale):
    """q [rows][H][d], k, v [rows][H_kv][d], sequence b in rows cu[b] .. cu[b+1]-1 -> (out, lse)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    rows, heads, d = q.shape
    group = heads // k.shape[1]
    out, lse = np.zeros((rows, heads, d)), np.zeros((rows, heads))
    for lo, hi in zip(cu[:-1], cu[1:]):
        for r in range(lo, hi):
            for h in range(heads):
                out[r, h], lse[r, h], _ = attention(q[r, h], k[lo:r + 1, h // group], v[lo:r + 1, h // group], scale)
    return out, lse
