"""CPU reference of decoding with drafted tokens, from the definitions: rotary positions, the attention of a
tree of drafts, the walk that keeps drafts, and the rows that stay. Plain Python and numpy in 64 bits (angles
and walks in exact rational arithmetic where asked)."""
import math
from fractions import Fraction

import numpy as np

# pi to 80 digits
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original=0, low=0.0, high=0.0, attention=0.0,
                     freqs=None):
    """(radians per position of each pair, factor of what is turned)."""
    out, a = [], 1.0
    for i in range(rot_dim // 2):
        if scaling == "given":
            out.append(float(freqs[i]))
            continue
        b = base * factor ** (rot_dim / (rot_dim - 2)) if scaling == "base" and rot_dim > 2 else base
        f = math.exp(-2 * i / rot_dim * math.log(b))
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = original * f / (2 * math.pi)              # within the original context
            if turns <= low:
                f /= factor
            elif turns < high:
                t = (turns - low) / (high - low)
                f = t * f + (1 - t) * f / factor
        elif scaling == "yarn":
            def pair(turns):
                return rot_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(0, math.floor(pair(high))), min(rot_dim - 1, math.ceil(pair(low)))
            t = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = t * f / factor + (1 - t) * f
            a = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
        out.append(f)
    return out, attention if attention > 0 else a


def rotate(x, positions, freqs, a, rot_dim, interleaved):
    """x [rows][heads][d] turned by integer positions; angles reduced in rational arithmetic."""
    y = np.array(x, dtype=np.float64)
    for p, f in enumerate(freqs):
        step = Fraction(f) / (2 * PI)
        turn = np.array([float((int(pos) * step) % 1) for pos in positions])
        c, s = a * np.cos(2 * math.pi * turn)[:, None], a * np.sin(2 * math.pi * turn)[:, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + rot_dim // 2)
        x1, x2 = np.array(x[..., i], dtype=np.float64), np.array(x[..., j], dtype=np.float64)
        y[..., i], y[..., j] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def tree_seen(n, t, row, bits=None):
    """Which of n tokens draft `row` of the last t sees: the prefix, and the drafts whose bit is set (None: up to its own)."""
    seen = np.ones(n, dtype=bool)
    for j in range(t):
        seen[n - t + j] = j <= row if bits is None else bool(bits >> j & 1)
    return seen


def tree_attend(q, k, v, seen, scale):
    """One query over the tokens it sees: (output, log sum exp, weights by token)."""
    w = np.zeros(len(k))
    if not seen.any():
        return np.zeros(v.shape[1]), -math.inf, w
    with np.errstate(all="ignore"):
        s = scale * (k[seen] @ q)
        m = s.max()
        e = np.exp(s - m)
        z = e.sum()
        w[seen] = e / z
        return (e / z) @ v[seen], m + math.log(z), w


def verify(tokens, parents, target, draft, u, u_next, distinct, number=float):
    """The walk over one sequence's tree: (nodes kept, token behind them). number: float, or Fraction for exact sums."""
    def at(rows, node, x):
        y = float(rows[node][x])
        return number(y) if y > 0 else number(0)

    def whole(node, c, gone):
        out = []
        for x in range(len(target[node])):
            p = at(target, node, x)
            if draft is not None:
                p = max(p - c * at(draft, node, x), number(0))
            elif x in gone:
                p = number(0)
            out.append(p)
        return out

    total = math.fsum if number is float else sum
    cur, path, c, z, w, gone = 0, [0], number(0), number(1), number(1), set()
    for i in range(1, len(tokens)):
        x = tokens[i]
        if not (0 <= parents[i] < i and 0 <= x < len(target[0])) or parents[i] != cur:
            continue
        if draft is not None:
            qx = at(draft, cur, x)
            yes = w > 0 and number(float(u[i])) * qx * z < max(at(target, cur, x) - c * qx, number(0)) * w
            if not yes:
                if w > 0:
                    c += z / w
                if distinct:
                    w -= qx
                z = total(whole(cur, c, gone))
        else:
            px = number(0) if x in gone else at(target, cur, x)
            yes = number(float(u[i])) * z < px
            if not yes:
                z -= px
                gone.add(x)
        if yes:
            cur, c, z, w, gone = i, number(0), number(1), number(1), set()
            path.append(i)
    r = whole(cur, c, gone)
    if not any(x > 0 for x in r):
        r = [at(target, cur, x) for x in range(len(target[cur]))]
    if not any(x > 0 for x in r):
        return path, -1
    t, run, last = number(float(u_next)) * total(r), number(0), -1
    for i, x in enumerate(r):
        run += x
        if x > 0:
            last = i
            if run > t:
                return path, i
    return path, last
