"""The history cache and the attention over it in float64 (test
infrastructure): what an 8-bit cache holds of a row, which events a row sees,
one row at a time, and O with the sums of absolute terms that error bounds are
stated in.
"""

from __future__ import annotations

import math

import numpy as np

from . import brute


def e4m3_values():
    """The 127 finite codes of one sign, in order (bias 7, subnormals, no infinity)."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m / 8.0 * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7))
    return np.array(out)


def row_exponent(top: float) -> int:
    """The least e >= -126 with top <= 448 * 2^e."""
    e = -126
    while top > math.ldexp(448.0, e):
        e += 1
    return e


def held(rows, store: str):
    """The values that a cache holds for float64 rows [..., d] (those of float32)."""
    if store != "e4m3":
        return rows.copy()
    codes = e4m3_values()
    out = np.empty_like(rows)
    for i in np.ndindex(rows.shape[:-1]):
        x = rows[i]
        if not np.all(np.isfinite(x)):
            out[i] = np.nan
            continue
        e = row_exponent(float(np.max(np.abs(x), initial=0.0)))
        y = np.ldexp(np.abs(x), -e)
        j = np.clip(np.searchsorted(codes, y), 1, 126)
        below, above = codes[j - 1], codes[j]
        # nearest, ties to the even code
        up = (y - below > above - y) | ((y - below == above - y) & (j % 2 == 0))
        up &= np.ldexp(above, e) < 2.0 ** 128      # codes whose value float32 does not hold
        out[i] = np.copysign(np.ldexp(np.where(up, above, below), e), x)
    return out


def sees(n: int, start: int, mask: str, window: int, sinks: int, parents=None):
    """[n, start + n] truth values: which events each of n new rows sees."""
    see = np.zeros((n, start + n), dtype=bool)
    place = list(range(start + n))
    see_all = np.zeros_like(see)   # the paths without the window
    for i in range(n):
        if mask == "history":
            path, p = set(range(start)), start
        elif mask == "causal":
            path, p = set(range(start + i + 1)), start + i
        else:
            up = int(parents[i])
            ok = 0 <= up < i
            path = set(np.flatnonzero(see_all[up])) if ok else set(range(start))
            path.add(start + i)
            p = place[start + up] + 1 if ok else start
            place[start + i] = p
        see_all[i, sorted(path)] = True
        for j in path:
            see[i, j] = window <= 0 or place[j] > p - window or place[j] < sinks
    return see


def attend(off, starts, q, k, v, alpha, act, mask="causal", window=0, sinks=0, parents=None):
    """q [T, H, d]; k, v: per sample float64 [events, Hkv, d] (what the cache
    holds).  (o, lse, size) as oracle.prefix.fwd's."""
    H = q.shape[1]
    o, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    size, size1, sizex = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    for b in range(len(off) - 1):
        n, s = int(off[b + 1] - off[b]), int(starts[b])
        rows = slice(int(off[b]), int(off[b + 1]))
        see = sees(n, s, mask, window, sinks, None if parents is None else parents[rows])
        rep = H // k[b].shape[1]
        for h in range(H):
            for i in range(n):
                on = np.flatnonzero(see[i])
                if not len(on):
                    continue
                t = int(off[b]) + i
                x = alpha * k[b][on, h // rep] @ q[t, h]
                val = v[b][on, h // rep]
                if act == "softmax":
                    top = x.max()
                    w = np.exp(x - top)
                    lse[t, h] = math.log(w.sum()) + top
                    w = w / w.sum()
                else:
                    w = brute.act(act, x)
                o[t, h] = w @ val
                size[t, h] = np.abs(w) @ np.abs(val)
                size1[t, h] = np.abs(val).sum(0)
                sizex[t, h] = np.abs(x) @ np.abs(val)
    return o, lse, (size, size1, sizex)
