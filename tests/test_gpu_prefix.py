"""Shared-prefix attention on the GPU against the float64 oracle: both kernel
families, forward and gradients.  Bounds: prefix_util (bf16: per value, from
the roundings; float32: 1e-5 of the largest value)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from prefix_util import batch, check_bf16, check_f32, check_lse, f64, orc, ref  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def setup_module(_):
    gd.build()


def make(offs, H, Hkv, d, dt, seed=0, gain=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rows(n, h, s):
        x = torch.randn((n, h, d), generator=g, device="cuda")
        return (x * (s * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6))).to(DT[dt])
    tq, tk, tp = int(offs[0][-1]), int(offs[1][-1]), int(offs[3][-1])
    return [rows(tq, H, gain), rows(tp, Hkv, 1.0), rows(tp, Hkv, 1.0), rows(tk, Hkv, 1.0),
            rows(tk, Hkv, 1.0), rows(tq, H, 1.0)]


def check(got, want, size, dt, act, name, slope=False):
    if dt == "f32":
        check_f32(got, want, name, size if slope else None)
    else:
        check_bf16(got, want, size, act, name, slope)


def run(offs, H, Hkv, d, dt, act, window=0, kernel="auto", backward=True, seed=0, num_sms=0,
        alpha=None, x=None):
    alpha = d ** -0.5 if alpha is None else alpha
    mask = "causal_window" if window else "none"
    x = make(offs, H, Hkv, d, dt, seed) if x is None else x
    plan = gd.PrefixPlan(*offs, H, d, kv_heads=Hkv, mask=mask, window=window, num_sms=num_sms)
    plan.set_kernel(kernel)
    y = f64(*x)
    if act == "softmax":
        o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5], alpha=alpha)
    else:
        o, lse = gd.gdpa_prefix_fwd(plan, *x[:5], act=act, alpha=alpha), None
    plan.check()
    want, wlse, size = orc.fwd(offs, *y[:5], alpha, act, mask, window)
    check(o, want, size, dt, act, "o")
    if lse is not None:
        check_lse(lse, wlse)
    if not backward:
        return plan, x, o, lse, None
    if act == "softmax":
        grads = gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse, alpha=alpha)
    else:
        grads = gd.gdpa_prefix_bwd(plan, *x[:5], x[5], act=act, alpha=alpha)
    plan.check()
    wg, sizes = orc.bwd(offs, *y, alpha, act, mask, window, ref.to_f64(o),
                        None if lse is None else ref.to_f64(lse))
    for name, g, w, s in zip(("dq", "dkp", "dvp", "dk", "dv"), grads, wg, sizes):
        check(g, w, s, dt, act, name, slope=name in ("dq", "dkp", "dk"))
    return plan, x, o, lse, grads


RAGGED = batch([3, 1, 0, 40, 2, 130, 1], [2, 0, 5, 40, 6, 131, 0], [2, 0, 3, 2], [4, 7, 0, 300])
SHAPES = {
    "ragged": RAGGED,
    "one token": batch([1], [0], [1], [1]),
    "no prefix": batch([5, 1], [7, 300], [2], [0]),
    "no keys": batch([5, 1], [0, 0], [1, 1], [0, 3]),
    "single tokens": batch([1] * 70, [i % 9 for i in range(70)], [1, 69], [1000, 257]),
    "two tiles": batch([257], [129], [1], [128]),
    "block edges": batch([127, 1, 128, 129], [127, 128, 129, 1], [2, 2], [129, 256]),
}


@pytest.mark.parametrize("dt,d,kernel", [("bf16", 128, "auto"), ("bf16", 64, "auto"),
                                         ("bf16", 128, "simt"), ("bf16", 40, "auto"),
                                         ("f32", 32, "auto"), ("f32", 128, "auto"), ("f32", 4, "auto")])
@pytest.mark.parametrize("act", ["softmax", "gelu_erf", "silu"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_shapes(shape, act, dt, d, kernel):
    run(SHAPES[shape], 2, 2, d, dt, act, kernel=kernel)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 20)])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (6, 2), (8, 4), (40, 1), (128, 1)])
def test_shared_key_heads(dt, d, H, Hkv):
    offs = batch([3, 1, 5, 2], [2, 0, 9, 130], [1, 3], [40, 200])
    run(offs, H, Hkv, d, dt, "softmax")
    run(offs, H, Hkv, d, dt, "gelu_tanh")


@pytest.mark.parametrize("dt,d,kernel", [("bf16", 128, "auto"), ("bf16", 64, "auto"),
                                         ("bf16", 64, "simt"), ("f32", 16, "auto")])
@pytest.mark.parametrize("window", [1, 20, 130, 2 ** 31 - 1])
@pytest.mark.parametrize("act", ["softmax", "silu"])
def test_windows(dt, d, kernel, window, act):
    """Rows behind the last own key see nothing of them; others a band."""
    offs = batch([300, 40, 7], [300, 10, 200], [2, 1], [0, 150])
    run(offs, 2, 1, d, dt, act, window=window, kernel=kernel)


@pytest.mark.parametrize("act", ["softmax", "gelu_erf", "gelu_tanh", "silu", "gelu_taylor6", "identity"])
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 64)])
def test_activations(act, dt, d):
    # queries small enough for the polynomial's range
    offs = batch([60, 10], [20, 3], [2], [150])
    x = make(offs, 2, 2, d, dt, gain=0.5)
    run(offs, 2, 2, d, dt, act, x=x)


@pytest.mark.parametrize("num_sms", [1, 2, 7, 152, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_queue_lengths(num_sms, d):
    """Few and many queues over the same batch: long walks and many parts."""
    offs = batch([200, 3, 1, 90], [64, 130, 0, 90], [1, 3], [1100, 640])
    run(offs, 4, 2, d, "bf16", "softmax", num_sms=num_sms)
    run(offs, 2, 2, d, "bf16", "silu", num_sms=num_sms)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_large_scores(dt, d):
    """Scores of hundreds: weights of one key per row, and sums that rise late."""
    offs = batch([50, 3], [33, 2], [2], [900])
    x = make(offs, 2, 2, d, dt)
    x[1] = (x[1].float() * torch.linspace(0.1, 30, 900, device="cuda")[:, None, None]).to(DT[dt])
    plan = gd.PrefixPlan(*offs, 2, d)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
    want, wlse, size = orc.fwd(offs, *f64(*x[:5]), d ** -0.5, "softmax")
    # a score of magnitude X has a float32 error of up to d 2^-24 X sqrt(d) here:
    # 128 * 2^-24 * 30 * 1.5 * 128 / sqrt(128) < 4e-3 of a weight
    err = np.abs(ref.to_f64(o) - want)
    slack = 4e-3 if dt == "bf16" else 4e-3
    assert np.all(err <= 1.02 * (2.0 ** -8 * np.abs(want) + 2.0 ** -8 * size[0]) + 2 * slack * size[0])
    assert np.max(np.abs(ref.to_f64(lse) - wlse) / np.maximum(1, np.abs(wlse))) < 2e-6


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_rows_next_to_a_key_range_do_not_leak(dt, d):
    """Infinities and NaN in the rows behind every prefix and every sample's own
    keys (which share 16-row and 128-row blocks with them) change nothing."""
    offs = batch([3, 2, 4], [5, 0, 17], [1, 2], [37, 130])
    x = make(offs, 2, 2, d, dt)
    plan = gd.PrefixPlan(*offs, 2, d)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
    # the same rows at other places, garbage between them
    gap = 19
    big = batch([3, 2, 4], [5, gap, 0, 17], [1, 3], [37, 130])
    k2, v2 = (torch.full((5 + gap + 17, 2, d), float("nan"), device="cuda").to(DT[dt]) for _ in "kv")
    for t, s in ((k2, x[3]), (v2, x[4])):
        t[:5], t[5 + gap:] = s[:5], s[5:]
        t[5:8] = float("inf")
    q_off = np.array([0, 3, 3, 5, 9], dtype=np.int32)
    kv_off = np.array([0, 5, 5 + gap, 5 + gap, 5 + gap + 17], dtype=np.int32)
    g_off, p_off = np.array([0, 1, 2, 4], dtype=np.int32), np.array([0, 37, 37 + gap, 167 + gap], dtype=np.int32)
    # group 1: a sample without queries owns the garbage keys and a garbage prefix
    kp2, vp2 = (torch.full((167 + gap, 2, d), float("inf"), device="cuda").to(DT[dt]) for _ in "kv")
    for t, s in ((kp2, x[1]), (vp2, x[2])):
        t[:37], t[37 + gap:] = s[:37], s[37:]
        t[37:40] = float("nan")
    plan2 = gd.PrefixPlan(q_off, kv_off, g_off, p_off, 2, d)
    o2, lse2 = gd.gdpa_prefix_softmax_fwd(plan2, x[0], kp2, vp2, k2, v2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g1 = gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse)
    g2 = gd.gdpa_prefix_softmax_bwd(plan2, x[0], kp2, vp2, k2, v2, o, x[5], lse)
    for a, b in zip((g2[0], g2[1][:37], g2[1][37 + gap:], g2[2][:37], g2[2][37 + gap:], g2[3][:5],
                     g2[3][5 + gap:], g2[4][:5], g2[4][5 + gap:]),
                    (g1[0], g1[1][:37], g1[1][37:], g1[2][:37], g1[2][37:], g1[3][:5], g1[3][5:],
                     g1[4][:5], g1[4][5:])):
        assert torch.isfinite(a).all()
        # dq may be summed in another order: a step of its rounding
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
    # keys that no query sees get no gradient
    for g in g2[1:3]:
        assert torch.all(g[37:37 + gap] == 0)
    for g in g2[3:]:
        assert torch.all(g[5:5 + gap] == 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_are_differences(dt):
    """<dO, O(x + e) - O(x - e)> / 2 against <grad, e>, float64 outside the kernels."""
    offs = batch([6, 3], [4, 2], [2], [50])
    d, H = 64, 2
    x = make(offs, H, H, d, "f32")
    if dt == "bf16":
        x = [t.bfloat16() for t in x]
    plan = gd.PrefixPlan(*offs, H, d)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
    grads = gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for i in range(5):
        e = torch.randn(x[i].shape, generator=g, device="cuda")
        h = 2.0 ** -6
        ys = [list(x), list(x)]
        ys[0][i], ys[1][i] = (x[i].float() + h * e).to(x[i].dtype), (x[i].float() - h * e).to(x[i].dtype)
        step = (ys[0][i].double() - ys[1][i].double())
        f = [(gd.gdpa_prefix_softmax_fwd(plan, *y[:5])[0].double() * x[5].double()).sum() for y in ys]
        got, want = float(f[0] - f[1]), float((grads[i].double() * step).sum())
        # O's and the gradient's own errors, as independent roundings; and the
        # cubic term of a step of 2^-6 in scores of a few units
        eps = 2.0 ** -8 if dt == "bf16" else 2.0 ** -18
        noise = eps * (float((o.double() * x[5].double()).square().sum().sqrt()) * 2 +
                       float((grads[i].double() * step).square().sum().sqrt())) * 4
        assert abs(got - want) <= noise + 2e-3 * abs(want) + 2e-3 * h, (i, got, want, noise)


def test_far_rows_past_32_bit_offsets():
    """Prefix rows whose byte and element offsets pass 2^32: the last group's
    prefix at the end of a tensor of 2^32 elements and more."""
    d, H = 128, 8
    n = 2 ** 22 + 300          # rows of 1024 elements
    kp = torch.zeros((n, H, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    offs = (np.array([0, 1, 4], dtype=np.int32), np.zeros(3, dtype=np.int32),
            np.array([0, 1, 2], dtype=np.int32), np.array([0, n - 200, n], dtype=np.int32))
    small = batch([3], [0], [1], [200])
    x = make(small, H, H, d, "bf16")
    kp[n - 200:], vp[n - 200:] = x[1], x[2]
    q = torch.cat([torch.zeros_like(x[0][:1]), x[0]])
    do = torch.cat([torch.zeros_like(x[5][:1]), x[5]])
    plan = gd.PrefixPlan(*offs, H, d)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, q, kp, vp)
    plan.check()
    want, wlse, size = orc.fwd(small, *f64(*x[:5]), d ** -0.5, "softmax")
    check_bf16(o[1:], want, size, "softmax", "o")
    assert torch.all(o[0] == 0) and abs(float(lse[0, 0]) - np.log(n - 200)) < 1e-5
    grads = gd.gdpa_prefix_softmax_bwd(plan, q, kp, vp, None, None, o, do, lse)
    plan.check()
    wg, sizes = orc.bwd(small, *f64(*x), d ** -0.5, "softmax", o=ref.to_f64(o[1:]), lse=ref.to_f64(lse[1:]))
    check_bf16(grads[1][n - 200:], wg[1], sizes[1], "softmax", "dkp", True)
    check_bf16(grads[2][n - 200:], wg[2], sizes[2], "softmax", "dvp")
    assert torch.all(grads[1][:n - 200] == 0)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 32)])
def test_streams_graphs_and_repeats(dt, d):
    offs = batch([5, 60, 1], [4, 70, 0], [2, 1], [300, 600])
    x = make(offs, 4, 2, d, dt)
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
    g = gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse)
    n = plan.launches
    assert n > 0
    # the forward gives the same bits again, on other streams in turn too
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [gd.gdpa_prefix_softmax_fwd(plan, *x[:5], stream=s[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)
    # a captured forward and backward, replayed on new inputs
    go, gl = torch.zeros_like(o), torch.zeros_like(lse)
    gg = [torch.zeros_like(t) for t in g]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gd.gdpa_prefix_softmax_fwd(plan, *x[:5], o=go, lse=gl)
        gd.gdpa_prefix_softmax_bwd(plan, *x[:5], go, x[5], gl, *gg)
    y = make(offs, 4, 2, d, dt, seed=7)
    for a, b in zip(x, y):
        a.copy_(b)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *y[:5])
    g = gd.gdpa_prefix_softmax_bwd(plan, *y[:5], o, y[5], lse)
    plan.check()
    assert torch.equal(go, o) and torch.equal(gl, lse)
    for a, b in zip(gg, g):   # float32 sums may come in another order before the rounding
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())


def test_first_backward_is_refused_while_capturing():
    offs = batch([5], [4], [1], [30])
    x = make(offs, 2, 2, 32, "f32")
    plan = gd.PrefixPlan(*offs, 2, 32)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
    out = [torch.empty_like(t) for t in x[:5]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(gd.GdpaError) as e:
            gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse, *out)
        out[0].zero_()   # the graph is not empty
    assert e.value.status == 4
    gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse, *out)   # and works outside


def test_together_with_rotary_positions():
    """Keys and queries turned by their positions (the prefix first, then the
    sample's rows), attention over both, and the gradients back through all."""
    offs = batch([4, 3, 6], [4, 3, 6], [2, 1], [70, 20])
    q_off, _, g_off, p_off = offs
    d, H = 32, 2
    x = make(offs, H, H, d, "f32")
    rope = gd.Rope(16, base=100.0)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    lp = np.diff(p_off)[np.searchsorted(g_off, np.arange(3), side="right") - 1]
    at = dict(offsets=dev(q_off), starts=dev(lp))
    q, k = gd.gdpa_rope_fwd(rope, x[0], x[3], **at)
    kp = gd.gdpa_rope_fwd(rope, x[1], offsets=dev(p_off))
    plan = gd.PrefixPlan(*offs, H, d, mask="causal_window", window=100)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, q, kp, x[2], k, x[4])
    dq, dkp, dvp, dk, dv = gd.gdpa_prefix_softmax_bwd(plan, q, kp, x[2], k, x[4], o, x[5], lse)
    dq, dk = gd.gdpa_rope_bwd(rope, dq, dk, **at)
    dkp = gd.gdpa_rope_bwd(rope, dkp, offsets=dev(p_off))
    from oracle import rope as orope
    f = orope.frequencies(16, base=100.0)
    y = f64(*x)
    pos_q = np.concatenate([n + np.arange(c) for n, c in zip(lp, np.diff(q_off))])
    pos_p = np.concatenate([np.arange(c) for c in np.diff(p_off)])
    tq, tk, tp = (orope.apply(a, p, f)[0] for a, p in ((y[0], pos_q), (y[3], pos_q), (y[1], pos_p)))
    a = d ** -0.5
    wo, wl, _ = orc.fwd(offs, tq, tp, y[2], tk, y[4], a, "softmax", "causal_window", 100)
    check_f32(o, wo, "o")
    check_lse(lse, wl)
    wg, _ = orc.bwd(offs, tq, tp, y[2], tk, y[4], y[5], a, "softmax", "causal_window", 100, wo, wl)
    for name, got, w, p in (("dq", dq, wg[0], pos_q), ("dk", dk, wg[3], pos_q), ("dkp", dkp, wg[1], pos_p)):
        check_f32(got, orope.apply(w, p, f, inverse=True)[0], name)
    check_f32(dvp, wg[2], "dvp")
    check_f32(dv, wg[4], "dv")


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 32), ("f32", 128)])
@pytest.mark.parametrize("act", ["softmax", "gelu_tanh"])
@pytest.mark.parametrize("shape", ["prefix", "two_prefixes", "own", "own_window"])
def test_many_rows_on_few_keys(shape, act, dt, d):
    """Key blocks whose rows are cut into ranges (more than six tiles of 128
    packed rows on a block, few blocks): the parts' sums, rows that end inside
    a tile, causal positions past a cut; and the same bits again."""
    offs, window = {
        "prefix": (batch([37] * 30, [5] * 30, [30], [70]), 0),
        "two_prefixes": (batch([40] * 21 + [3] * 2, [0] * 23, [21, 2], [1, 130]), 0),
        "own": (batch([1100, 7], [150, 2], [1, 1], [3, 0]), 0),
        "own_window": (batch([1500], [200], [1], [3]), 700),
    }[shape]
    H, Hkv = 4, 1
    plan, x, o, lse, grads = run(offs, H, Hkv, d, dt, act, window=window)
    kw = dict(alpha=d ** -0.5)
    again = (gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse, **kw) if act == "softmax"
             else gd.gdpa_prefix_bwd(plan, *x[:5], x[5], act=act, **kw))
    for a, b in zip(grads, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
def test_rows_aligned_to_16_bytes_only(dt, d):
    """Every tensor 16 bytes past a 32-byte boundary: the same bits."""
    H, Hkv = 4, 2
    plan, x, o, lse, grads = run(RAGGED, H, Hkv, d, dt, "softmax")

    def moved(t):
        step = 16 // t.element_size()
        y = torch.empty(t.numel() + 2 * step, dtype=t.dtype, device="cuda")
        at = step if y.data_ptr() % 32 == 0 else 2 * step
        y = y[at:at + t.numel()].view(t.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(t)
    kw = dict(alpha=d ** -0.5)
    m = [moved(t) for t in x]
    o2, _ = gd.gdpa_prefix_softmax_fwd(plan, *m[:5], o=moved(o), **kw)
    outs = dict(zip(("dq", "dkp", "dvp", "dk", "dv"), (moved(g).fill_(7.0) for g in grads)))
    got = gd.gdpa_prefix_softmax_bwd(plan, *m[:5], moved(o), m[5], lse, **outs, **kw)
    assert torch.equal(o2, o)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt,d,kernel", [("bf16", 128, "auto"), ("bf16", 64, "auto"), ("f32", 32, "auto"),
                                         ("bf16", 128, "simt")])
@pytest.mark.parametrize("key", [0, 3, 4, 5, 130])
def test_nan_scores_reach_the_rows_that_see_them(dt, d, kernel, key):
    """A NaN key makes O and lse NaN for exactly the rows that see it: of a
    group (prefix), or of a sample (its only own key, and one of many)."""
    lq, lkv = [3, 1, 9, 70], [1, 0, 200, 140]
    offs = batch(lq, lkv, [2, 2], [150, 0])
    x = make(offs, 2, 2, d, dt)
    plan = gd.PrefixPlan(*offs, 2, d)
    plan.set_kernel(kernel)
    first, q_off = int(offs[1][2]), offs[0]
    for where, row, rows in (("prefix", key, (0, 4)), ("only own", 0, (0, 3)), ("small own", first + key, (4, 13)),
                             ("own", int(offs[1][3]) + key, (13, 83))):
        y = [t.clone() for t in x]
        y[1 if where == "prefix" else 3][row, 1] = float("nan")
        o, lse = gd.gdpa_prefix_softmax_fwd(plan, *y[:5])
        seen = torch.zeros(83, 2, dtype=torch.bool, device="cuda")
        seen[rows[0]:rows[1], 1] = True
        assert torch.equal(torch.isnan(lse), seen), where
        assert torch.equal(torch.isnan(o).all(-1), seen) and torch.equal(torch.isnan(o).any(-1), seen), where


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("alpha", [0.0, -0.125])
def test_scales_of_zero_and_below(alpha, act, dt, d):
    run(RAGGED, 4, 2, d, dt, act, window=3, alpha=alpha)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("offs", [batch([], [], [], []), batch([0, 0], [40, 0], [1, 1], [5, 300]),
                                  batch([2], [0], [1], [0])])
def test_nothing_to_do(offs, dt, d):
    """No samples; keys without rows (gradients of zeros); rows without keys."""
    plan, x, o, lse, grads = run(offs, 2, 2, d, dt, "softmax")
    assert torch.all(o == 0) and torch.all(lse == -float("inf"))
    for g in grads:
        assert torch.all(g == 0)


def test_two_host_threads_share_a_plan():
    import threading
    offs = batch([5, 60, 1], [4, 70, 0], [2, 1], [300, 600])
    d = 128
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    x = [make(offs, 4, 2, d, "bf16", seed=i) for i in range(2)]
    want = []
    for y in x:
        o, lse = gd.gdpa_prefix_softmax_fwd(plan, *y[:5])
        want.append((o, gd.gdpa_prefix_softmax_bwd(plan, *y[:5], o, y[5], lse)))
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        y, st = x[i], torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(10):
                o, lse = gd.gdpa_prefix_softmax_fwd(plan, *y[:5])
                got[i].append((o, gd.gdpa_prefix_softmax_bwd(plan, *y[:5], o, y[5], lse)))
        st.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 10
        for o, g in got[i]:
            assert torch.equal(o, want[i][0])
            for a, b in zip(g, want[i][1]):
                assert torch.equal(a, b)


def test_refusals():
    offs = batch([5], [4], [1], [30])
    x = make(offs, 2, 2, 32, "f32")
    plan = gd.PrefixPlan(*offs, 2, 32)
    q, kp, vp, k, v, do = x
    for bad in ((q[:4], kp, vp, k, v), (q, kp[:4], vp, k, v), (q, kp, vp, None, None),
                (q.cpu(), kp, vp, k, v), (q, kp, vp, k, v[:, :1]),
                (q, kp.transpose(0, 1).contiguous().transpose(0, 1), vp, k, v)):
        with pytest.raises((ValueError, AttributeError)):
            gd.gdpa_prefix_softmax_fwd(plan, *bad)
    for bad in ((q, kp.bfloat16(), vp, k, v), tuple(t.half() for t in x[:5])):
        with pytest.raises(TypeError):
            gd.gdpa_prefix_softmax_fwd(plan, *bad)
    with pytest.raises(ValueError):
        gd.gdpa_prefix_softmax_fwd(plan, q, kp, vp, k, v, lse=torch.empty((5, 2), device="cuda").half())
    with pytest.raises(ValueError):
        gd.gdpa_prefix_bwd(plan, q, kp, vp, k, v, do, act="softmax")
    with pytest.raises(KeyError):
        gd.gdpa_prefix_fwd(plan, q, kp, vp, k, v, act="relu")
    plan.set_kernel("tcgen05")   # float32 has none
    with pytest.raises(gd.GdpaError) as e:
        gd.gdpa_prefix_softmax_fwd(plan, q, kp, vp, k, v)
    assert e.value.status == 2
    plan.set_kernel("auto")
    # misaligned rows
    w = torch.empty(q.numel() + 1, device="cuda")[1:].view(q.shape)
    with pytest.raises(gd.GdpaError) as e:
        gd.gdpa_prefix_softmax_fwd(plan, w, kp, vp, k, v)
    assert e.value.status == 1
    plan.destroy()
    with pytest.raises(RuntimeError):
        gd.gdpa_prefix_softmax_fwd(plan, q, kp, vp, k, v)
