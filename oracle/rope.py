"""Rotary positions in exact arithmetic and float64 (test infrastructure).

Angles are reduced with integers: a float64 frequency is a rational number,
and 1 / (2 pi) is taken to 60 digits, so the fraction of a turn at any 64-bit
position is right to far beyond float64.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

# 1 / (2 pi)
INV_TWO_PI = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


def frequencies(n, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, lo=1.0, hi=32.0):
    """Radians per position of each of the n / 2 pairs (float64)."""
    if scaling == "ntk" and n > 2:
        base = base * factor ** (n / (n - 2.0))
    out = []
    for i in range(n // 2):
        f = base ** (-2.0 * i / n)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            g = (orig_len * f / (2.0 * math.pi) - lo) / (hi - lo)
            g = min(1.0, max(0.0, g))
            f = g * f + (1.0 - g) * f / factor
        out.append(f)
    return np.array(out)


def turns_fixed(f) -> int:
    """f / (2 pi) modulo one turn in units of 2^-64 turns, to nearest."""
    x = Fraction(float(f)) * INV_TWO_PI * 2 ** 64
    return int(math.floor(abs(x) + Fraction(1, 2))) * (1 if x >= 0 else -1) % 2 ** 64


def cos_sin(positions, freqs):
    """cos and sin of position * frequency, [T, n / 2] each (float64)."""
    c = np.empty((len(positions), len(freqs)))
    s = np.empty_like(c)
    for j, f in enumerate(freqs):
        per = Fraction(float(f)) * INV_TWO_PI
        for i, p in enumerate(positions):
            t = (per * int(p)) % 1
            a = 2.0 * math.pi * float(t if t <= Fraction(1, 2) else t - 1)
            c[i, j], s[i, j] = math.cos(a), math.sin(a)
    return c, s


def apply(x, positions, freqs, layout="half", scale=1.0, inverse=False):
    """Turned rows of x ([T, heads, d] float64) and, per value, |a| + |b| of its
    pair (0 where nothing turns), which error bounds are stated in."""
    x = np.asarray(x, dtype=np.float64)
    n = 2 * len(freqs)
    c, s = cos_sin(positions, freqs)
    c, s = c[:, None] * scale, s[:, None] * (-scale if inverse else scale)
    ia = np.arange(n // 2) if layout == "half" else 2 * np.arange(n // 2)
    ib = ia + n // 2 if layout == "half" else ia + 1
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size
