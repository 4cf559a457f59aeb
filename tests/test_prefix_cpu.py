"""Shared-prefix attention without a GPU: the oracle's pins, what the plan
covers, and the refusals."""

import ctypes

import numpy as np
import pytest

import recommender_model_attention_gb300 as gd
from oracle import brute
from prefix_util import batch, orc


def setup_module(_):
    gd.build()


def _case(seed, lq, lkv, cand, lp, H, Hkv, d):
    rng = np.random.default_rng(seed)
    offs = batch(lq, lkv, cand, lp)
    tq, tk, tp = int(offs[0][-1]), int(offs[1][-1]), int(offs[3][-1])
    r = lambda n, h: rng.standard_normal((n, h, d)) * 0.7  # noqa: E731
    return offs, r(tq, H), r(tp, Hkv), r(tp, Hkv), r(tk, Hkv), r(tk, Hkv), r(tq, H)


LQ, LKV, CAND, LP = [3, 1, 0, 4, 2], [2, 0, 5, 3, 6], [2, 0, 3], [4, 7, 0]


@pytest.mark.parametrize("act", ["softmax", "gelu_erf", "gelu_taylor6", "identity"])
def test_oracle_is_attention_over_the_repeated_prefix(act):
    """Repeating the prefix in front of every sample's own keys gives the dense
    padded form's problem."""
    offs, q, kp, vp, k, v, do = _case(0, LQ, LKV, CAND, LP, 2, 2, 4)
    q_off, kv_off, g_off, p_off = offs
    ks, vs, n = [], [], []
    for b in range(len(LQ)):
        g = int(np.searchsorted(g_off, b, side="right")) - 1
        pre, own = slice(p_off[g], p_off[g + 1]), slice(kv_off[b], kv_off[b + 1])
        ks += [kp[pre], k[own]]
        vs += [vp[pre], v[own]]
        n.append(p_off[g + 1] - p_off[g] + LKV[b])
    full = np.concatenate([[0], np.cumsum(n)])
    want = brute.fwd(q_off, full, q, np.concatenate(ks), np.concatenate(vs), 0.5, act)
    got, lse, _ = orc.fwd(offs, q, kp, vp, k, v, 0.5, act)
    assert np.allclose(got, want, atol=1e-13)


@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("mask,window", [("none", 0), ("causal_window", 2)])
def test_oracle_gradients_are_differences(act, mask, window):
    offs, *x, do = _case(1, LQ, LKV, CAND, LP, 4, 2, 4)
    alpha = 0.4
    o, lse, _ = orc.fwd(offs, *x, alpha, act, mask, window)
    grads, _ = orc.bwd(offs, *x, do, alpha, act, mask, window, o, lse)
    rng = np.random.default_rng(2)
    for i, g in enumerate(grads):
        e = rng.standard_normal(x[i].shape)
        f = []
        for s in (1e-5, -1e-5):
            y = list(x)
            y[i] = x[i] + s * e
            f.append((orc.fwd(offs, *y, alpha, act, mask, window)[0] * do).sum())
        assert (f[0] - f[1]) / 2e-5 == pytest.approx((g * e).sum(), rel=1e-6, abs=1e-8)


def _covered(plan, offs, H, Hkv, window):
    """Every (query row, key) that a row sees is in exactly one part."""
    q_off, kv_off, g_off, p_off = offs
    r, tpt = H // Hkv, 128 // (H // Hkv)
    pieces, seg = plan.export()
    assert seg[0] == 0 and np.all(np.diff(seg) >= 0) and seg[-1] <= len(pieces)
    assert np.all(pieces[seg[-1]:, 6] & 1)   # behind the queues: small own pieces only
    pre = np.zeros((plan.Tq, Hkv, plan.Tp), dtype=np.int8)
    own = np.zeros((plan.Tq, Hkv, max(1, plan.Tkv)), dtype=np.int8)
    parts = []
    for tok, na, nb, hk, k0, nk, flags, i0, j0, pa, pb, _ in pieces.tolist():
        assert 0 < na <= tpt and 0 <= nb <= tpt and nk > 0
        to = own if flags & 1 else pre
        if flags & 2:
            assert nb == 0 and (pb >= 0) == (nk > 128)
        to[tok:tok + na + nb, hk, k0:k0 + nk] += 1
        parts += [(p, n * r) for p, n in ((pa, na), (pb, na if flags & 2 else nb)) if p >= 0]
        if flags & 1:
            b = int(np.searchsorted(q_off, tok, side="right")) - 1
            assert tok == q_off[b] + i0 and k0 == kv_off[b] + j0
    parts.sort()   # rows of the workspace: one part behind the other
    assert [p for p, _ in parts] == np.cumsum([0] + [n for _, n in parts]).tolist()[:-1]
    for rows, p, o, see in orc.groups(*offs, "causal_window" if window else "none", window):
        for hk in range(Hkv):
            assert np.all(pre[rows][:, hk][:, p] == 1)
            cover = own[rows][:, hk][:, o] if len(o) else np.zeros((len(rows), 0))
            assert np.all(cover <= 1) and np.all(cover >= see[:, len(p):])
    assert pre.sum() == sum((q_off[g_off[g + 1]] - q_off[g_off[g]]) * (p_off[g + 1] - p_off[g])
                            for g in range(plan.G)) * Hkv
    return pieces, seg


@pytest.mark.parametrize("lq,lkv,cand,lp", [
    (LQ, LKV, CAND, LP), ([1], [0], [1], [1]), ([1], [1], [1], [0]), ([0], [0], [1], [5]),
    ([1] * 16, [0] * 16, [16], [2000]), ([1] * 150, [3] * 150, [150], [513]),
    ([300, 1], [290, 140], [1, 1], [129, 700]), ([40] * 9, [40] * 9, [4, 5], [256, 1000]),
    ([], [], [], []), ([], [], [0, 0], [9, 0])])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 2), (128, 1), (4, 4)])
@pytest.mark.parametrize("window,sms", [(0, 1), (0, 152), (37, 5)])
def test_plan_covers_every_pair_once(lq, lkv, cand, lp, H, Hkv, window, sms):
    offs = batch(lq, lkv, cand, lp)
    plan = gd.PrefixPlan(*offs, H, 8, kv_heads=Hkv, mask="causal_window" if window else "none",
                         window=window, num_sms=sms, host_only=True)
    _covered(plan, offs, H, Hkv, window)


def test_plan_balances_and_spreads():
    """A short batch against a long prefix reaches every SM, and no share of a
    ragged one is far above the mean."""
    one = batch([1] * 16, [0] * 16, [16], [65536])
    plan = gd.PrefixPlan(*one, 4, 128, num_sms=152, host_only=True)
    pieces, seg = _covered(plan, one, 4, 4, 0)
    assert np.count_nonzero(np.diff(seg)) >= 140
    rng = np.random.default_rng(0)
    cand, lp = rng.integers(1, 100, 30), rng.integers(1, 3000, 30)
    offs = batch(np.ones(cand.sum(), int), np.zeros(cand.sum(), int), cand, lp)
    plan = gd.PrefixPlan(*offs, 8, 128, num_sms=152, host_only=True)
    pieces, seg = plan.export()
    steps = -(-pieces[:, 5] // np.where(pieces[:, 6] & 2, 256, 128)) + 3
    load = np.add.reduceat(np.append(steps, 0), np.minimum(seg[:-1], len(steps)))[np.diff(seg) > 0]
    assert load.max() <= 1.25 * (steps.sum() / 152) + 4


@pytest.mark.parametrize("kw,status", [
    (dict(H=0), 1), (dict(kv_heads=0), 1), (dict(kv_heads=3), 1), (dict(d=130), 2), (dict(d=6), 2),
    (dict(d=132), 2), (dict(H=256, kv_heads=1), 2), (dict(H=1 << 18, d=8, kv_heads=1 << 18), 2),
    (dict(mask="causal_window", window=0), 1), (dict(num_sms=0), 1), (dict(num_sms=-1), 1),
    (dict(q_off=[1, 2]), 1), (dict(q_off=[0, -1]), 1), (dict(kv_off=[0, -4]), 1),
    (dict(group_off=[0, 2]), 1), (dict(group_off=[0, 0]), 1), (dict(prefix_off=[3, 4]), 1)])
def test_refused_plans(kw, status):
    a = dict(q_off=[0, 2], kv_off=[0, 2], group_off=[0, 1], prefix_off=[0, 4], H=4, d=64, kv_heads=2,
             num_sms=4)
    a.update(kw)
    with pytest.raises(gd.GdpaError) as e:
        gd.PrefixPlan(host_only=True, **a)
    assert e.value.status == status


def test_refused_shapes_and_host_plans():
    with pytest.raises(ValueError):
        gd.PrefixPlan([0, 1], [0], [0, 1], [0, 1], 1, 8, num_sms=1, host_only=True)
    with pytest.raises(ValueError):
        gd.PrefixPlan([0, 1], [0, 1], [0, 1], [0], 1, 8, num_sms=1, host_only=True)
    plan = gd.PrefixPlan([0, 1], None, [0, 1], [0, 1], 1, 8, num_sms=1, host_only=True)
    L, f = gd.lib(), ctypes.c_float(1.0)
    p = 4096
    assert L.gdpa_prefix_fwd(plan.handle, 0, p, p, p, None, None, p, None, f, 5, 0) == 1
    assert L.gdpa_prefix_bwd(plan.handle, 0, p, p, p, None, None, p, p, p, p, p, p, None, None, f, 5, 0) == 1
    assert L.gdpa_prefix_check(plan.handle, 0) == 1
    assert L.gdpa_prefix_fwd(None, 0, p, p, p, None, None, p, None, f, 5, 0) == 1
    assert L.gdpa_prefix_set_kernel(plan.handle, 3) == 1 and L.gdpa_prefix_set_kernel(plan.handle, 2) == 0
    assert L.gdpa_prefix_launches(None) == -1 and plan.launches == 0
    L.gdpa_prefix_destroy(None)
    plan.destroy()
    plan.destroy()
    with pytest.raises(RuntimeError):
        plan.export()
