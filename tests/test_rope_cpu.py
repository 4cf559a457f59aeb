"""Rotary positions without a GPU: the frequency table's bits, the oracle's
own pins, and the refusals of the C entry points."""

import ctypes
import math

import numpy as np
import pytest

import recommender_model_attention_gb300 as gd
from oracle import rope as orc
from recommender_model_attention_gb300 import gdpa as raw


def setup_module(_):
    gd.build()


def _turns(r):
    return [int(r.spec.turns[i]) for i in range(r.rot_dim // 2)]


def test_inv_two_pi_is_the_reciprocal_of_two_pi():
    # Machin: pi / 4 = 4 atan(1/5) - atan(1/239), in 80-digit integers
    one = 10 ** 80

    def atan_inv(n):
        total, term, k = 0, one // n, 0
        while term:
            total += term // (2 * k + 1) * (-1 if k & 1 else 1)
            term //= n * n
            k += 1
        return total
    pi = 4 * (4 * atan_inv(5) - atan_inv(239))
    assert abs(int(orc.INV_TWO_PI * one) * 2 * pi // one - one) < 10 ** 22


@pytest.mark.parametrize("f", [1.0, -1.0, 0.0, 1e-4, 0.75, 6.283185307179586, 1048576.0, -1048576.0,
                               3.0 / 7, 1e-19, 2.0 ** -62, 2.0 ** -63, 1e-30, 5e-324, 12345.678])
def test_turns_are_exact_to_the_last_bit(f):
    r = gd.Rope(2, freqs=[f])
    got, want = _turns(r)[0], orc.turns_fixed(f)
    # one unit (2^-64 turns): the library's constant has 128 bits
    assert min((got - want) % 2 ** 64, (want - got) % 2 ** 64) <= (1 if abs(f) > 1e-6 else 0), (got, want)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
@pytest.mark.parametrize("n", [2, 6, 64, 128])
def test_scaled_frequencies(scaling, n):
    kw = dict(base=50000.0, scaling=scaling, factor=3.0, orig_len=512.0, lo=1.0, hi=8.0)
    r = gd.Rope(n, **kw)
    want = orc.frequencies(n, **kw)
    for got, f in zip(_turns(r), want):
        # pow differs between maths libraries by an ulp or two; the table's
        # entry is rounded to a unit of 2^-64, half of which is 2^-65
        assert abs(got / 2.0 ** 64 - f / (2 * math.pi)) <= 8 * 2.0 ** -53 * f + 2.0 ** -65
    if scaling == "by_parts" and n >= 64:   # the ends of the ramp are both met
        plain = orc.frequencies(n, base=50000.0)
        assert want[0] == plain[0] and want[-1] == pytest.approx(plain[-1] / 3.0, rel=1e-15)


def test_oracle_turns_keep_length_and_distance():
    rng = np.random.default_rng(0)
    f = orc.frequencies(16)
    x = rng.standard_normal((5, 2, 20))
    y, _ = orc.apply(x, [0, 1, 7, 10 ** 9, -3], f)
    assert np.allclose((y[..., :16] ** 2).sum(-1), (x[..., :16] ** 2).sum(-1), rtol=1e-13)
    assert np.array_equal(y[..., 16:], x[..., 16:]) and np.array_equal(y[0], x[0])
    back, _ = orc.apply(y, [0, 1, 7, 10 ** 9, -3], f, inverse=True)
    assert np.allclose(back, x, atol=1e-14)
    # q at p and k at p' depend on p - p' alone
    q, k = x[0:1], x[1:2]
    dots = [(orc.apply(q, [a], f)[0] * orc.apply(k, [b], f)[0]).sum()
            for a, b in ((5, 2), (10 ** 9 + 3, 10 ** 9), (0, -3))]
    assert np.ptp(dots) < 1e-12


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=-2),
                                dict(rot_dim=4, base=0.5), dict(rot_dim=4, base=math.inf),
                                dict(rot_dim=4, scaling="linear", factor=0.5),
                                dict(rot_dim=4, scaling="by_parts", factor=2.0),
                                dict(rot_dim=4, scaling="by_parts", factor=2.0, orig_len=9, lo=2, hi=2),
                                dict(rot_dim=4, scale=math.nan),
                                dict(rot_dim=4, freqs=[1.0, math.nan]),
                                dict(rot_dim=4, freqs=[1.0, 2e6])])
def test_refused_tables(kw):
    with pytest.raises(gd.GdpaError) as e:
        gd.Rope(**kw)
    assert e.value.status == 1


def test_refused_sizes():
    with pytest.raises(gd.GdpaError) as e:
        gd.Rope(130)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        gd.Rope(4, freqs=[1.0])
    with pytest.raises(KeyError):
        gd.Rope(4, layout="diagonal")


def _apply(rope, dtype=0, T=4, d=8, heads=2, n=1, pos=64, bits=32, off=0, B=0, x=4096, tok=16, head=8):
    rows = 2 * raw._rope_tensor(x, x, heads, tok, head, tok, head)
    return gd.lib().gdpa_rope_apply(ctypes.byref(rope.spec), 0, dtype, T, d, rows, n, pos, bits, off,
                                    0, B, 0)


def test_refused_calls():
    """Every refusal comes before any launch (there is no GPU here)."""
    half, inter = gd.Rope(8), gd.Rope(8, layout="interleaved")
    for kw in (dict(dtype=7), dict(T=-1), dict(d=6), dict(n=0), dict(n=3), dict(heads=-1),
               dict(x=0), dict(x=4097), dict(bits=16), dict(pos=0), dict(pos=0, off=64, B=-1),
               dict(pos=64, off=64), dict(pos=66, bits=32), dict(pos=68, bits=64)):
        assert _apply(half, **kw) == 1, kw
    assert _apply(half, d=130) == 2
    assert _apply(half, heads=5000) == 2
    for kw in (dict(d=9), dict(tok=17), dict(head=9), dict(x=4098)):
        assert _apply(inter, **kw) == 1, kw
    # nothing to do: no launch, no error
    assert _apply(half, T=0) == 0 and _apply(half, heads=0) == 0
