"""Pins of the drafted-token oracle and of the host part of rotary positions: known values, and properties that
the definitions must have. No GPU."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import token_level_sparse_gb300 as T
from oracle import draft_oracle as D

CASES = [dict(rot_dim=128, base=10000.0), dict(rot_dim=2, base=10000.0), dict(rot_dim=64, base=500000.0, scaling="linear", factor=4.0),
         dict(rot_dim=128, base=10000.0, scaling="base", factor=8.0), dict(rot_dim=2, scaling="base", factor=8.0),
         dict(rot_dim=128, base=500000.0, scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0),
         dict(rot_dim=128, base=1000000.0, scaling="yarn", factor=4.0, original=32768, low=1.0, high=32.0),
         dict(rot_dim=22, base=10000.0, scaling="yarn", factor=40.0, original=4096, low=1.0, high=32.0, attention=0.5),
         dict(rot_dim=6, scaling="given", freqs=[1.0, -0.25, 7.5])]


@pytest.fixture(scope="module")
def lib():
    from token_level_sparse_gb300 import build
    build.build()
    return T.library()


@pytest.mark.parametrize("case", CASES)
def test_frequencies_of_a_handle(lib, case):
    want, a = D.rope_frequencies(**case)
    got, b = T.Rope(**case).read()
    # pow and exp(log) of 64 bits: an error of the logarithm (below 14) grows to 14 ulps of the result and some roundings
    assert np.allclose(got, want, rtol=64 * 2.0 ** -52, atol=0) and abs(a - b) <= 2.0 ** -24 * a


def test_frequencies_by_hand():
    f, a = D.rope_frequencies(4, base=100.0)
    assert f[0] == 1.0 and abs(f[1] - 0.1) < 1e-15 and a == 1.0
    # within 1000 positions the pairs turn 159, 15.9 and 1.59 times: kept, between, scaled
    f, _ = D.rope_frequencies(6, base=1000.0, scaling="bands", factor=10.0, original=1000, low=2.0, high=100.0)
    t = (100 / (2 * math.pi) - 2) / 98
    assert abs(f[0] - 1.0) < 1e-12 and abs(f[1] - (0.1 * t + 0.01 * (1 - t))) < 1e-12 and abs(f[2] - 0.001) < 1e-15


def test_rotation_by_hand_and_back():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y = D.rotate(x, [1], [math.pi / 2, math.pi], 1.0, 4, False)
    assert np.allclose(y, [[[-3.0, -2.0, 1.0, -4.0, 5.0]]])
    y = D.rotate(x, [1], [math.pi / 2, math.pi], 2.0, 4, True)
    assert np.allclose(y, [[[-4.0, 2.0, -6.0, -8.0, 5.0]]])
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 8))
    pos = np.array([0, 1, 77, 10 ** 6, 2 ** 31 - 1])
    f, _ = D.rope_frequencies(8)
    assert np.allclose(D.rotate(D.rotate(x, pos, f, 1.0, 8, False), -pos, f, 1.0, 8, False), x, atol=1e-12)


def test_bad_handles_are_refused(lib):
    bad = [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=130), dict(rot_dim=8, base=0.0), dict(rot_dim=8, base=math.nan),
           dict(rot_dim=8, scaling="linear", factor=0.0), dict(rot_dim=8, scaling="bands", factor=2.0, original=0, low=1.0, high=4.0),
           dict(rot_dim=8, scaling="bands", factor=2.0, original=100, low=4.0, high=4.0), dict(rot_dim=8, attention=-1.0),
           dict(rot_dim=8, scaling="yarn", base=1.0, factor=2.0, original=100, low=1.0, high=4.0), dict(rot_dim=8, scaling="none"),
           dict(rot_dim=4, scaling="given", freqs=[1.0, math.inf]), dict(rot_dim=4, scaling="given", freqs=[1.0]),
           dict(rot_dim=4, scaling="given"), dict(rot_dim=4, scaling="plain", freqs=[1.0, 1.0])]
    for case in bad:
        with pytest.raises(T.TokenSelectError):
            T.Rope(**case)
    INVALID = T.STATUS_CODE["TS_ERR_INVALID_ARG"]
    assert lib.ts_rope_create(None, None) == INVALID and lib.ts_rope_destroy(None) == INVALID
    assert lib.ts_rope_read(None, None, None) == INVALID
    cfg = T.RopeConfig(8, 2, 0, 10000.0)
    h = ctypes.c_void_p()
    assert lib.ts_rope_create(ctypes.byref(h), ctypes.byref(cfg)) == INVALID and not h.value


def test_null_arguments_are_refused(lib):
    INVALID = T.STATUS_CODE["TS_ERR_INVALID_ARG"]
    assert lib.ts_rotate(None, None, None, 0, 0, 0, None, 0, None, 0, 0, None) == INVALID
    assert lib.ts_append_rotated(None, None, None, 0, None, 0, None, None, None, 0, 0, None, None, None, None, 0, None, 0, 0, None) == INVALID
    assert lib.ts_tree_attend(None, None, 0, None, None, None, None, None, None, 0, 0, 0, 0.0, None, 0, None, None) == INVALID
    assert lib.ts_verify_tree(None, None, None, None, 0, 0, 0, None, 0, None, 0, None, None, 0, None, 0, None, None, None) == INVALID
    assert lib.ts_keep_rows(None, None, 0, None, None, None, 0, 0, None, None, None, 0, 0, None, None) == INVALID


# ------------------------------------------------------------------- the walk

def test_walk_by_hand():
    p = [[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]]
    q = [[0.25, 0.5, 0.25], [0.5, 0.5, 0.0], [0.25, 0.5, 0.25]]
    # token 1 drafted twice at the root: u q = 0.3 is not below 0.25; then r = (0.25, 0, 0), nothing left for token 1
    assert D.verify([9, 1, 1], [-1, 0, 0], p, q, [0, 0.6, 0.1], 0.9, False) == ([0], 0)
    # taken at once, then a chain: behind node 1 token 1 is certain
    assert D.verify([9, 1, 1], [-1, 0, 1], p, q, [0, 0.4, 0.9], 0.5, False) == ([0, 1, 2], 2)
    # greedy drafts: 0.6 refuses token 0 (0.5); of what is left token 2 has half: 0.4 * 0.5 < 0.25 takes it
    assert D.verify([9, 0, 2], [-1, 0, 0], p, None, [0, 0.6, 0.4], 0.0, False) == ([0, 2], 0)
    # everything refused: drawn from what is left
    assert D.verify([9, 0, 2], [-1, 0, 0], p, None, [0, 0.6, 0.6], 0.9, False) == ([0], 1)
    # bad nodes are passed over; a row without mass ends in -1
    assert D.verify([9, 3, 1], [-1, 0, 2], p, q, [0, 0, 0], 0.0, False) == ([0], 0)
    assert D.verify([9], [-1], [[0.0, math.nan, -1.0]], None, [0], 0.0, False) == ([0], -1)


@pytest.mark.parametrize("distinct,greedy", [(False, False), (True, False), (False, True)])
def test_tokens_come_out_as_the_target_has_them(distinct, greedy):
    """The token behind the root, whichever way it was found, has the target's distribution: exactly, by adding up the
    probability of every outcome over a grid-free enumeration: the drafts' draws, then the walk's uniform numbers."""
    p = [Fraction(x, 20) for x in (8, 1, 6, 5)]
    q = [Fraction(x, 20) for x in (2, 9, 4, 5)]
    out = [Fraction(0)] * 4

    def walk(c, z, w, r, left, weight, gone):
        """Distribution of the emitted token when `left` children are still to come; r unnormalised, its sum z."""
        if left == 0:
            s = sum(r)
            for i in range(4):
                out[i] += weight * r[i] / s
            return
        for x in range(4):
            if greedy:
                pick = Fraction(int(x == [1, 2, 0][3 - left]))
                take = r[x] / z if pick else Fraction(0)
            else:
                pick = (Fraction(0) if distinct and x in gone else q[x] / (w if distinct else 1))
                take = min(Fraction(1), r[x] * w / (q[x] * z)) if pick else Fraction(0)
            if not pick:
                continue
            out[x] += weight * pick * take
            if take == 1:
                continue
            if greedy:
                r2 = [Fraction(0) if i == x else r[i] for i in range(4)]
                walk(c, z - r[x], w, r2, left - 1, weight * pick * (1 - take), gone | {x})
            else:
                c2 = c + z / w
                r2 = [max(p[i] - c2 * q[i], Fraction(0)) for i in range(4)]
                if not any(r2):
                    r2 = p
                walk(c2, sum(r2), w - (q[x] if distinct else 0), r2, left - 1, weight * pick * (1 - take), gone | {x})

    walk(Fraction(0), Fraction(1), Fraction(1), p, 3, Fraction(1), frozenset())
    assert out == p


def test_exact_and_float_walks_agree():
    rng = np.random.default_rng(3)
    for case in range(60):
        V, n = int(rng.integers(2, 12)), int(rng.integers(1, 10))
        p, q = (rng.dirichlet(np.full(V, 0.5), size=n).astype(np.float32) for _ in range(2))
        par = [-1] + [int(rng.integers(0, i)) for i in range(1, n)]
        tok = [int(x) for x in rng.integers(0, V, n)]
        u, un = rng.random(n).astype(np.float32), np.float32(rng.random())
        for distinct in (False, True):
            for draft in (q, None):
                assert D.verify(tok, par, p, draft, u, un, distinct) == D.verify(tok, par, p, draft, u, un, distinct, Fraction)


def test_tree_attention_by_hand():
    k = np.array([[0.0], [math.log(3.0)], [5.0]])
    v = np.array([[1.0], [2.0], [math.nan]])
    seen = D.tree_seen(3, 2, 0)
    assert seen.tolist() == [True, True, False]
    out, lse, w = D.tree_attend(np.array([1.0]), k, v, seen, 1.0)
    assert np.allclose(out, [1.75]) and np.isclose(lse, math.log(4.0)) and w[2] == 0
    assert D.tree_seen(3, 2, 1, bits=0b10).tolist() == [True, False, True]
    out, lse, _ = D.tree_attend(np.array([1.0]), k, v, D.tree_seen(3, 3, 1, bits=0), 1.0)
    assert out.tolist() == [0.0] and lse == -math.inf
