"""Outputs that a call allocates for another stream than the current one: their
memory must not be in use yet by work queued on the current stream, nor be given
out again before its uses there are over."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402

pytestmark = pytest.mark.gpu

T, H, D = 600, 4, 128


def setup_module(_):
    gd.build()


def _calls():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    q, k, v = (torch.randn((T, H, D), generator=g, device="cuda").bfloat16() for _ in range(3))
    off = np.array([0, 200, T], dtype=np.int32)
    plan = gd.Plan(off, off, H, D)
    prefix = gd.PrefixPlan(off, off, [0, 2], [0, T], H, D)
    rope, pos = gd.Rope(D), torch.arange(T, device="cuda")
    o, lse = gd.gdpa_prefix_softmax_fwd(prefix, q, k, v, k, v)
    return {
        "rope": lambda **kw: gd.gdpa_rope_fwd(rope, q, k, positions=pos, **kw),
        "prefix": lambda **kw: gd.gdpa_prefix_softmax_fwd(prefix, q, k, v, k, v, **kw),
        "prefix_bwd": lambda **kw: gd.gdpa_prefix_softmax_bwd(prefix, q, k, v, k, v, o, q, lse, **kw),
        "gdpa": lambda **kw: (gd.gdpa_fwd(plan, q, k, v, act="silu", **kw),),
        # dK and dV: GDPA's dQ is added up atomically, in an order that may change
        "gdpa_bwd": lambda **kw: gd.gdpa_bwd(plan, q, k, v, q, act="silu", **kw)[1:],
        "softmax": lambda **kw: gd.gdpa_softmax_fwd(plan, q, k, v, **kw),
        "mx": lambda **kw: tuple(gd.mx_quantise(q, **kw)),
    }


@pytest.mark.parametrize("name", ["rope", "prefix", "prefix_bwd", "gdpa", "gdpa_bwd", "softmax", "mx"])
def test_outputs_of_a_call_on_another_stream(name):
    call = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed with writes to them still to come on
    # the current stream
    junk = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(50_000_000)
    for t in junk:
        t.fill_(7)
    del junk, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # freed with reads of them still to come on the current stream
    torch.cuda._sleep(50_000_000)
    copies = [a.clone() for a in got]
    sizes = [(a.shape, a.dtype) for a in got]
    del got, a
    with torch.cuda.stream(side):
        more = [torch.full(shape, 7, dtype=dt, device="cuda") for shape, dt in sizes]
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
    del more


@pytest.mark.parametrize("name", ["rope", "prefix", "prefix_bwd"])
def test_outputs_allocated_for_another_stream_of_a_capture(name):
    """A captured call on a branch of the graph that allocates its outputs."""
    call = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):   # outputs freed while capturing, then some that are kept
            got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(2):
        for t in copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, copies, want):
            assert torch.equal(a, c) and torch.equal(b, c)
