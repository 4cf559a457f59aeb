"""Shared-prefix attention on the GPU at the edges of what its calls allow:
what the window hides, streams, captures and limits.  Helpers and bounds as
test_gpu_prefix.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from prefix_util import batch, f64, orc, ref  # noqa: E402
from test_gpu_prefix import DT, make, run  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 128, "auto"), ("bf16", 64, "auto"), ("bf16", 128, "simt"), ("bf16", 64, "simt"),
         ("f32", 32, "auto")]


def setup_module(_):
    gd.build()


def both(plan, x, act):
    """Forward and gradients: a list of tensors."""
    if act == "softmax":
        o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
        out = [o, lse, *gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse)]
    else:
        out = [gd.gdpa_prefix_fwd(plan, *x[:5], act=act), *gd.gdpa_prefix_bwd(plan, *x[:5], x[5], act=act)]
    plan.check()
    return out


def garbage(t, rows):
    """t with infinities and NaN in turn in the given rows."""
    t = t.clone()
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        t[rows[i::3]] = bad
    return t


@pytest.mark.parametrize("dt,d,kernel", KINDS)
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("window", [1, 5, 100, 2 ** 31 - 1])
def test_keys_hidden_from_all_rows_may_hold_anything(window, act, dt, d, kernel):
    """Own keys behind their sample's last row, in samples of up to 8, up to 64
    and more packed rows: the same bits whatever they hold, gradients of 0."""
    lq, lkv = [2, 1, 4, 20, 32, 130, 6], [40, 9, 17, 60, 300, 200, 6]
    offs = batch(lq, lkv, [3, 4], [37, 0])
    x = make(offs, 2, 1, d, dt)
    plan = gd.PrefixPlan(*offs, 2, d, kv_heads=1, mask="causal_window", window=window)
    plan.set_kernel(kernel)
    rows = torch.from_numpy(np.concatenate(
        [np.arange(offs[1][b] + min(lq[b], lkv[b]), offs[1][b + 1]) for b in range(len(lq))])).cuda()
    want = both(plan, x, act)
    got = both(plan, [x[0], x[1], x[2], garbage(x[3], rows), garbage(x[4], rows), x[5]], act)
    for a, b in zip(got, want):
        assert torch.isfinite(b).all() and torch.equal(a, b)
    for g in got[-2:]:
        assert torch.all(g[rows] == 0)


@pytest.mark.parametrize("dt,d,kernel", KINDS)
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("window", [1, 3])
def test_rows_that_see_no_key_may_hold_anything(window, act, dt, d, kernel):
    """Query rows behind the last own key's window, in groups without a prefix:
    they leave every gradient as it is and have none."""
    lq, lkv = [4, 30, 200, 3], [1, 3, 5, 3]
    offs = batch(lq, lkv, [2, 2], [0, 0])
    x = make(offs, 2, 1, d, dt)
    plan = gd.PrefixPlan(*offs, 2, d, kv_heads=1, mask="causal_window", window=window)
    plan.set_kernel(kernel)
    rows = torch.from_numpy(np.concatenate(
        [np.arange(offs[0][b] + min(lq[b], lkv[b] + window - 1), offs[0][b + 1]) for b in range(len(lq))])).cuda()
    assert len(rows) > 100
    want = both(plan, x, act)
    got = both(plan, [garbage(x[0], rows), *x[1:5], garbage(x[5], rows)], act)
    for i, (a, b) in enumerate(zip(got, want)):
        if act == "softmax" and i == 1:
            assert torch.all(a[rows] == -float("inf"))
        else:
            assert torch.isfinite(b).all()
        assert torch.equal(a, b)
    assert torch.all(got[0][rows] == 0) and torch.all(got[-5][rows] == 0)


class PerThread:
    """The per-thread default stream: one handle, another stream in each thread."""
    cuda_stream = 2


def test_threads_on_the_per_thread_stream_share_a_plan():
    """Two host threads, each on its own per-thread default stream (equal
    handles), forward and backward on one plan and different inputs: the
    workspace is one, so the calls have to follow one another on the GPU."""
    import threading
    offs = batch([5, 300, 1], [4, 310, 0], [2, 1], [2000, 9000])
    d = 128
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    x = [make(offs, 4, 2, d, "bf16", seed=i) for i in range(2)]
    want = [both(plan, y, "softmax") for y in x]
    # a turn of outputs per call, made here: allocations belong to a stream
    outs = [[[torch.zeros_like(t) for t in want[i]] for _ in range(20)] for i in range(2)]
    torch.cuda.synchronize()
    meet, failed = threading.Barrier(2), []

    def work(i):
        try:
            meet.wait(60)
            y = x[i]
            for o, lse, *g in outs[i]:
                gd.gdpa_prefix_softmax_fwd(plan, *y[:5], o=o, lse=lse, stream=PerThread)
                gd.gdpa_prefix_softmax_bwd(plan, *y[:5], o, y[5], lse, *g, stream=PerThread)
            # (a thread's exit destroys its stream, which must not have work left)
            torch.cuda.ExternalStream(PerThread.cuda_stream).synchronize()
        except Exception as e:   # noqa: BLE001  (shown below)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,), daemon=True) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and not any(t.is_alive() for t in threads), failed
    torch.cuda.synchronize()
    plan.check()
    for i in range(2):
        for call in outs[i]:
            for a, b in zip(call, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 32)])
def test_calls_on_two_streams_of_one_capture(dt, d):
    """Forwards and backwards of different inputs on two branches of a captured
    graph share the plan's workspace: every replay gives each its own results."""
    offs = batch([5, 300, 1], [4, 310, 0], [2, 1], [2000, 9000])
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    x = [make(offs, 4, 2, d, dt, seed=i) for i in range(2)]
    want = [both(plan, y, "softmax") for y in x]
    outs = [[torch.zeros_like(t) for t in want[i]] for i in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for part in ("fwd", "bwd"):
            for i, stream in enumerate((None, side)):
                o, lse, *g = outs[i]
                if part == "fwd":
                    gd.gdpa_prefix_softmax_fwd(plan, *x[i][:5], o=o, lse=lse, stream=stream)
                else:
                    gd.gdpa_prefix_softmax_bwd(plan, *x[i][:5], o, x[i][5], lse, *g, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(10):
        for call in outs:
            for t in call:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(a, b)
    # another capture of the plan, and eager calls, afterwards
    again = torch.cuda.CUDAGraph()
    o, lse, *g = outs[0]
    with torch.cuda.graph(again):
        gd.gdpa_prefix_softmax_fwd(plan, *x[0][:5], o=o, lse=lse)
    o.zero_()
    again.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0])
    for a, b in zip(both(plan, x[1], "softmax"), want[1]):
        assert torch.equal(a, b)


def test_plans_are_refused_on_a_stream_that_is_captured():
    offs = batch([5], [4], [1], [30])
    x = make(offs, 2, 2, 64, "bf16")
    out = torch.zeros(3, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(gd.GdpaError) as e:
            gd.PrefixPlan(*offs, 2, 64)
        out.fill_(2)   # the capture goes on
    assert e.value.status == 4
    graph.replay()
    torch.cuda.synchronize()
    assert torch.all(out == 2)
    both(gd.PrefixPlan(*offs, 2, 64), x, "softmax")


@pytest.mark.parametrize("d", [32, 128])
def test_large_scores_float32(d):
    """Scores of hundreds in float32, to a bound that weights or rows rounded to
    bf16 would break.

    A score is d products summed in float32, off by at most d 2^-24 of its
    absolute terms A, and its scale's product by 2^-24 of it: e = (d + 1) 2^-24
    max_j A_ij for a row i.  The weights over their sum are then off by a factor
    of e^(2 e), and by what exp (2 ulp), the 900 sums of weights and values and
    the joining of parts add, below 1000 * 2^-24 of the absolute sum together."""
    offs = batch([50, 3], [33, 2], [2], [900])
    x = make(offs, 2, 2, d, "f32")
    x[1] = x[1] * torch.linspace(0.1, 30, 900, device="cuda")[:, None, None]
    plan = gd.PrefixPlan(*offs, 2, d)
    o, lse = gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
    plan.check()
    y = f64(*x[:5])
    want, wlse, size = orc.fwd(offs, *y, d ** -0.5, "softmax")
    terms = np.zeros(wlse.shape)
    for rows, pre, own, see in orc.groups(*offs):
        for h in range(2):
            a = np.abs(y[0][rows, h]) @ np.abs(np.concatenate([y[1][pre, h], y[3][own, h]])).T * d ** -0.5
            terms[rows, h] = np.where(see, a, 0.0).max(1)
    e = (d + 1) * 2.0 ** -24 * terms
    assert wlse.max() > 50
    err = np.abs(ref.to_f64(o) - want)
    bound = (np.exp(2 * e) - 1 + 1000 * 2.0 ** -24)[..., None] * size[0]
    assert np.all(err <= bound), np.max(err / bound)
    assert np.all(np.abs(ref.to_f64(lse) - wlse) <= e + 1000 * 2.0 ** -24 + 2.0 ** -22 * np.abs(wlse))
    # the bound sees a rounding to bf16: the plain form with bf16 rows breaks it
    r = [ref.to_f64(t.bfloat16()) for t in x[:5]]
    assert np.any(np.abs(orc.fwd(offs, *r, d ** -0.5, "softmax")[0] - want) > bound)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", range(4, 129, 4))
def test_every_head_dim(d, dt):
    offs = batch([3, 1, 0, 40], [2, 0, 5, 40], [2, 2], [4, 70])
    run(offs, 2, 1, d, dt, "softmax", window=7)


@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 32)])
def test_outputs_over_inputs(dt, d, act):
    """o and dq may be an input's memory, being stored last; key gradients, which
    are stored while keys are still read, are refused there and over each other."""
    offs = batch([5, 60, 1], [4, 70, 0], [2, 1], [300, 600])
    x = make(offs, 4, 2, d, dt)
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    want = both(plan, x, act)
    sm = act == "softmax"
    o, lse = want[0], want[1] if sm else None

    def bwd(y, do, o=o, **kw):
        if sm:
            return gd.gdpa_prefix_softmax_bwd(plan, *y, o, do, lse, **kw)
        return gd.gdpa_prefix_bwd(plan, *y, do, act=act, **kw)
    for name in ("q", "do", "o"):
        y, do, o2 = [t.clone() for t in x[:5]], x[5].clone(), o.clone()
        got = bwd(y, do, o2, dq={"q": y[0], "do": do, "o": o2}[name])
        for a, b in zip(got, want[-5:]):
            assert torch.equal(a, b)
    q = x[0].clone()
    if sm:
        got = gd.gdpa_prefix_softmax_fwd(plan, q, *x[1:5], o=q)[0]
    else:
        got = gd.gdpa_prefix_fwd(plan, q, *x[1:5], act=act, o=q)
    assert torch.equal(got, o)
    spare = torch.zeros(2 * x[1].numel(), dtype=x[1].dtype, device="cuda")
    half = x[1].numel() - 64   # (a multiple of 16 bytes)
    over = dict(dkp=spare[:x[1].numel()].view(x[1].shape), dvp=spare[half:half + x[1].numel()].view(x[1].shape))
    for kw in (dict(dk=x[3]), dict(dv=x[4]), dict(dkp=x[1]), dict(dvp=x[2]), dict(dkp=x[2]), dict(dv=x[3]), over,
               dict(dk=torch.empty_like(x[3]), dv=None)):
        if kw.get("dv", 0) is None:
            kw["dv"] = kw["dk"]
        with pytest.raises(gd.GdpaError) as e:
            bwd(x[:5], x[5], **kw)
        assert e.value.status == 1
    for a, b in zip(both(plan, x, act), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt,H,kernel", [("bf16", 8, "auto"), ("f32", 8, "auto"), ("bf16", 8, "simt")])
def test_far_own_keys_past_32_bit_offsets(dt, H, kernel):
    """Own keys whose element and byte offsets pass 2^32: a small sample, one of
    9 to 64 rows and a large one behind a sample without rows that owns 2^22 keys."""
    d, n = 128, 2 ** 22
    lq, lkv = [0, 2, 30, 100], [n, 40, 50, 90]
    offs, small = batch(lq, lkv, [4], [60]), batch(lq[1:], lkv[1:], [3], [60])
    x = make(small, H, H, d, dt)
    alone = gd.PrefixPlan(*small, H, d)
    alone.set_kernel(kernel)
    want = both(alone, x, "softmax")
    k, v = (torch.zeros((n + 180, H, d), dtype=DT[dt], device="cuda") for _ in "kv")
    k[n:], v[n:] = x[3], x[4]
    plan = gd.PrefixPlan(*offs, H, d)
    plan.set_kernel(kernel)
    got = both(plan, [x[0], x[1], x[2], k, v, x[5]], "softmax")
    for a, b in zip(got[5:], want[5:]):
        assert torch.all(a[:n] == 0)
        # (pieces are dealt to the queues in other places: other parts' sums)
        assert float((a[n:].float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
    for a, b in zip(got[:5], want[:5]):
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())


def test_two_captures_under_way_at_once():
    """Calls of two captures alternate; each capture has two branches, so a call
    has to find the plan's call before it in its own."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.13")

    def ok(e):
        assert e == 0, e
    offs = batch([5, 300, 1], [4, 310, 0], [2, 1], [2000, 9000])
    d = 128
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    x = [make(offs, 4, 2, d, "bf16", seed=i) for i in range(4)]
    want = [both(plan, y, "softmax") for y in x]
    outs = [[torch.zeros_like(t) for t in want[i]] for i in range(4)]
    main, side, event = ([torch.cuda.Stream() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)],
                         [[ctypes.c_void_p() for _ in range(2)] for _ in range(2)])
    torch.cuda.synchronize()
    for m, s, e in zip(main, side, event):   # (relaxed: allocations elsewhere do not end them)
        for one in e:
            ok(rt.cudaEventCreateWithFlags(ctypes.byref(one), 2))
        ok(rt.cudaStreamBeginCapture(ctypes.c_void_p(m.cuda_stream), 2))
        ok(rt.cudaEventRecord(e[0], ctypes.c_void_p(m.cuda_stream)))
        ok(rt.cudaStreamWaitEvent(ctypes.c_void_p(s.cuda_stream), e[0], 0))
    for part in ("fwd", "bwd"):
        for branch in range(2):
            for c in range(2):
                i = 2 * c + branch
                o, lse, *g = outs[i]
                st = (main, side)[branch][c]
                if part == "fwd":
                    gd.gdpa_prefix_softmax_fwd(plan, *x[i][:5], o=o, lse=lse, stream=st)
                else:
                    gd.gdpa_prefix_softmax_bwd(plan, *x[i][:5], o, x[i][5], lse, *g, stream=st)
    graphs = []
    for m, s, e in zip(main, side, event):
        graph, run_it = ctypes.c_void_p(), ctypes.c_void_p()
        ok(rt.cudaEventRecord(e[1], ctypes.c_void_p(s.cuda_stream)))
        ok(rt.cudaStreamWaitEvent(ctypes.c_void_p(m.cuda_stream), e[1], 0))
        ok(rt.cudaStreamEndCapture(ctypes.c_void_p(m.cuda_stream), ctypes.byref(graph)))
        ok(rt.cudaGraphInstantiate(ctypes.byref(run_it), graph, ctypes.c_ulonglong(0)))
        graphs.append((graph, run_it))
    for _ in range(10):
        for call in outs:
            for t in call:
                t.zero_()
        torch.cuda.synchronize()
        for _, run_it in graphs:   # one after the other
            ok(rt.cudaGraphLaunch(run_it, ctypes.c_void_p(main[0].cuda_stream)))
        torch.cuda.synchronize()
        for i in range(4):
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(a, b)
    for graph, run_it in graphs:
        ok(rt.cudaGraphExecDestroy(run_it))
        ok(rt.cudaGraphDestroy(graph))
    for e in event:
        for one in e:
            ok(rt.cudaEventDestroy(one))


def test_more_captures_than_are_remembered():
    offs = batch([5, 60, 1], [4, 70, 0], [2, 1], [300, 600])
    x = make(offs, 4, 2, 64, "bf16")
    plan = gd.PrefixPlan(*offs, 4, 64, kv_heads=2)
    want = both(plan, x, "softmax")
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    for _ in range(40):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gd.gdpa_prefix_softmax_fwd(plan, *x[:5], o=o, lse=lse)
            gd.gdpa_prefix_softmax_fwd(plan, *x[:5], o=o, lse=lse)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0])
