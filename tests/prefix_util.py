"""Cases and error bounds of shared-prefix attention, for its CPU and GPU tests."""

import numpy as np

from oracle import prefix as orc
from oracle import ref

# Errors of the tensor-core kernels' activations (csrc/act.cuh): a fit of
# GELU-erf within 3.4e-4 (value) and 6.7e-4 (slope), and tanh.approx within
# 2^-11, which enters the value as |x| / 2 and the slope as 1/2 + 1.2 |x|.
ACT_ERR = {"gelu_erf": ((3.4e-4, 2.0 ** -12), (6.7e-4 + 2.0 ** -12, 1.2 * 2.0 ** -11)),
           "gelu_tanh": ((0.0, 2.0 ** -12), (2.0 ** -12, 1.2 * 2.0 ** -11)),
           "silu": ((0.0, 2.0 ** -12), (2.0 ** -12, 1.2 * 2.0 ** -11))}


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def batch(lq, lkv, cand, lp):
    """(q_off, kv_off, group_off, prefix_off) from lengths."""
    return offsets(lq), offsets(lkv), offsets(cand), offsets(lp)


def bound_of(want, size, kind, act, slope=False):
    """Largest error of a bf16 result: half a bf16 step (2^-8) of the value for
    its own rounding and of every term for the rounding of its weight, 2^-12 of
    every term for the float32 sums behind the weight, and the activation's
    error; 2% for products of these."""
    terms, one, x = size
    c1, cx = ACT_ERR.get(act, ((0.0, 0.0), (0.0, 0.0)))[1 if slope else 0]
    return 1.02 * (2.0 ** -8 * np.abs(want) + 2.0 ** -8 * terms + c1 * one + cx * x) + 1e-30


def check_bf16(got, want, size, act, name, slope=False):
    err = np.abs(ref.to_f64(got) - want)
    b = bound_of(want, size, name, act, slope)
    assert np.all(err <= b), "%s: worst error %.3g of its bound" % (name, np.max(err / b))


def check_f32(got, want, name, size=None):
    """The float32 bound of the attention kernels, 1e-5 of the largest value;
    for gradients (size given) beside it the float32 error of dS = p (dP - D),
    whose terms cancel (a row with one key has dS = 0): a sum of d products is
    off by at most d 2^-24 of its absolute terms, D and the subtraction add a
    few more, and size[0] holds 2^-4 of those terms: (d + 8) 2^-20 size[0]."""
    top = np.max(np.abs(want)) if want.size else 0.0
    b = 1e-5 * top + 1e-30
    if size is not None:
        b = b + (want.shape[-1] + 8) * 2.0 ** -20 * size[0]
    err = np.abs(ref.to_f64(got) - want)
    assert np.all(err <= b), "%s: %.3g of its bound" % (name, np.max(err / b))


def check_lse(got, want):
    """lse to 1e-5 absolute (float32) of a sum of scores of at most a few tens."""
    g = ref.to_f64(got)
    assert np.array_equal(np.isinf(g), np.isinf(want)) and np.array_equal(g[np.isinf(g)], want[np.isinf(want)])
    ok = np.isfinite(want)
    if ok.any():
        assert np.max(np.abs(g[ok] - want[ok]) / np.maximum(1.0, np.abs(want[ok]))) <= 2e-6


def f64(*ts):
    return [ref.to_f64(t) for t in ts]


__all__ = ["batch", "offsets", "check_bf16", "check_f32", "check_lse", "f64", "orc", "ref"]
