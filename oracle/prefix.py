"""Shared-prefix attention in float64 (test infrastructure): group by group
with the keys a group's rows can see side by side and an explicit mask, one
query head at a time.  Beside every result stands the sum of the absolute
values of its terms, in which error bounds are stated.
"""

from __future__ import annotations

import numpy as np

from . import brute


def groups(q_off, kv_off, group_off, prefix_off, mask="none", window=0):
    """Per group: (query rows, prefix rows, own rows, mask [rows, prefix + own])."""
    for g in range(len(group_off) - 1):
        b0, b1 = int(group_off[g]), int(group_off[g + 1])
        rows = np.arange(q_off[b0], q_off[b1])
        pre = np.arange(prefix_off[g], prefix_off[g + 1])
        own = np.arange(kv_off[b0], kv_off[b1])
        see = np.zeros((len(rows), len(pre) + len(own)), dtype=bool)
        see[:, :len(pre)] = True
        for b in range(b0, b1):
            for i in range(int(q_off[b + 1] - q_off[b])):
                for j in range(int(kv_off[b + 1] - kv_off[b])):
                    ok = mask == "none" or (j <= i and j > i - window)
                    see[q_off[b] - q_off[b0] + i, len(pre) + kv_off[b] - kv_off[b0] + j] = ok
        yield rows, pre, own, see


def _weights(x, see, act):
    """Weights of one head's scores x = alpha q.k, and the row log-sum-exp."""
    if act != "softmax":
        return np.where(see, brute.act(act, x), 0.0), None
    x = np.where(see, x, -np.inf)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = x.max(axis=1, initial=-np.inf)
        e = np.exp(x - np.where(np.isfinite(top), top, 0.0)[:, None])
        s = e.sum(1)
        lse = np.where(s > 0, np.log(s) + top, -np.inf)
        return e / np.where(s > 0, s, 1.0)[:, None], lse


def fwd(offs, q, kp, vp, k, v, alpha, act, mask="none", window=0):
    """(o, lse, size): size = sum of |w| |V| (element-wise acts: + what an
    error of one unit in every weight adds, as size1)."""
    H, Hkv = q.shape[1], kp.shape[1]
    o, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    size, size1, sizex = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    for rows, pre, own, see in groups(*offs, mask, window):
        for h in range(H):
            e = h // (H // Hkv)
            key = np.concatenate([kp[pre, e], k[own, e]])
            val = np.concatenate([vp[pre, e], v[own, e]])
            if not len(rows) or not len(key):
                continue
            x = alpha * q[rows, h] @ key.T
            w, l = _weights(x, see, act)
            o[rows, h] = w @ val
            size[rows, h] = np.abs(w) @ np.abs(val)
            size1[rows, h] = see @ np.abs(val)
            sizex[rows, h] = np.where(see, np.abs(x), 0.0) @ np.abs(val)
            if l is not None:
                lse[rows, h] = l
    return o, lse, (size, size1, sizex)


def bwd(offs, q, kp, vp, k, v, do, alpha, act, mask="none", window=0, o=None, lse=None):
    """Gradients (dq, dkp, dvp, dk, dv) and, for each, its absolute sums with
    every factor's own absolute terms: (rounded weights, weight slope errors)."""
    H, Hkv = q.shape[1], kp.shape[1]
    names = ("dq", "dkp", "dvp", "dk", "dv")
    like = (q, kp, vp, k, v)
    out = {n: np.zeros_like(x) for n, x in zip(names, like)}
    size = {n: [np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)] for n, x in zip(names, like)}
    for rows, pre, own, see in groups(*offs, mask, window):
        np_ = len(pre)
        for h in range(H):
            e = h // (H // Hkv)
            key = np.concatenate([kp[pre, e], k[own, e]])
            val = np.concatenate([vp[pre, e], v[own, e]])
            if not len(rows) or not len(key):
                continue
            x = alpha * q[rows, h] @ key.T
            dout = do[rows, h]
            dp, dpa = dout @ val.T, np.abs(dout) @ np.abs(val).T
            if act == "softmax":
                l = lse[rows, h][:, None]
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.where(see & np.isfinite(l), np.exp(x - np.where(np.isfinite(l), l, 0.0)), 0.0)
                delta = (dout * o[rows, h]).sum(1, keepdims=True)
                deltaa = np.abs(dout * o[rows, h]).sum(1, keepdims=True)
                ds, dsa = p * (dp - delta), p * (dpa + deltaa)
            else:
                p = np.where(see, brute.act(act, x), 0.0)
                slope = brute.dact(act, x)
                ds = np.where(see, slope * dp, 0.0)
                dsa = np.where(see, np.abs(slope) * dpa, 0.0)
            one = see.astype(np.float64)
            xa = np.where(see, np.abs(x), 0.0)
            # (value, rounding of the weights, float32 terms, error of a unit
            # in act or act', of |x| in it)
            terms = {"q": (ds, np.abs(ds), dsa, one * np.abs(dp), xa * np.abs(dp)),
                     "p": (p, np.abs(p), np.abs(p), one, xa)}
            q_, d_ = np.abs(q[rows, h]), np.abs(dout)

            def add(n, at, t, a, b, scale):
                w, wr, wf, w1, wx = terms[t]
                out[n][at, h if n == "dq" else e] += scale * a(w, b)
                for i, m in enumerate((wr + 2.0 ** -4 * wf, w1, wx)):
                    size[n][i][at, h if n == "dq" else e] += abs(scale) * a(m, np.abs(b))
            add("dq", rows, "q", lambda w, b: w @ b, key, alpha)
            left = lambda s: (lambda w, b: w[:, s].T @ b)  # noqa: E731
            P, O = slice(0, np_), slice(np_, None)
            add("dkp", pre, "q", left(P), q[rows, h], alpha)
            add("dk", own, "q", left(O), q[rows, h], alpha)
            add("dvp", pre, "p", left(P), dout, 1.0)
            add("dv", own, "p", left(O), dout, 1.0)
    return [out[n] for n in names], [size[n] for n in names]
