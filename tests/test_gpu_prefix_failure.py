"""Failure path of the shared-prefix tensor-core kernels, without a GPU fault.

Every barrier wait is bounded.  The plan's test hook shortens the limit to 20 ms
and makes CTA 0 of one kernel skip its first query load, so that a wait for it
is never satisfied: the kernel must record a timeout, unwind (its copies and
products in flight finish, TMEM is freed) and return, check() must report
GDPA_ERR_TIMEOUT with the place, and the next call on the plan must be right.
"""

import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from prefix_util import batch  # noqa: E402
from test_gpu_prefix import make, run  # noqa: E402

pytestmark = pytest.mark.gpu

TIMEOUT = 5   # GDPA_ERR_TIMEOUT
# wait sites of the forward, the dK, dV kernel and the dQ kernel
SITES = {"fwd": range(61, 74), "dkv": range(81, 93), "dq": range(101, 113)}


def setup_module(_):
    gd.build()


@pytest.mark.parametrize("which", ["fwd", "dkv", "dq"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("size", ["long", "one tile"])
def test_expired_wait_reports_timeout_and_plan_recovers(size, act, d, which):
    # queues longer than the rings of loads; and one piece and unit, of few keys
    offs = {"long": batch([300, 200, 2], [290, 200, 0], [2, 1], [3000, 40000]),
            "one tile": batch([5], [0], [1], [100])}[size]
    x = make(offs, 4, 2, d, "bf16")
    plan = gd.PrefixPlan(*offs, 4, d, kv_heads=2)
    pieces = gd.PrefixPlan(*offs, 4, d, kv_heads=2, num_sms=152, host_only=True)
    assert pieces.export()[1][1] > 0 and pieces.export_list("unit_seg")[1, 0] > 0   # CTA 0 has work

    def fwd():
        if act == "softmax":
            return gd.gdpa_prefix_softmax_fwd(plan, *x[:5])
        return gd.gdpa_prefix_fwd(plan, *x[:5], act=act), None

    def bwd(o, lse):
        if act == "softmax":
            return gd.gdpa_prefix_softmax_bwd(plan, *x[:5], o, x[5], lse)
        return gd.gdpa_prefix_bwd(plan, *x[:5], x[5], act=act)
    o, lse = fwd()
    grads = bwd(o, lse)
    plan.check()
    assert plan.error_detail() == (0, 0, 0, 0)
    plan.set_wait_test(limit_us=20000, stall=2 if which == "dq" else 1)
    t0 = time.time()
    if which == "fwd":
        fwd()
    else:
        bwd(o, lse)
    with pytest.raises(gd.GdpaError) as e:
        plan.check()
    assert e.value.status == TIMEOUT
    code, site, cta, _ = plan.error_detail()
    assert code == 1 and cta == 0 and site in SITES[which], plan.error_detail()
    assert time.time() - t0 < 10.0   # well inside the default limit (2 s a wait)
    # reported once; the next calls on the plan are right
    plan.set_wait_test()
    plan.check()
    o2, lse2 = fwd()
    again = bwd(o2, lse2)
    plan.check()
    assert torch.equal(o2, o) and (lse is None or torch.equal(lse2, lse))
    for a, b in zip(again, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [128, 64])
def test_results_next_to_the_hook_are_the_oracles(d):
    """The batch of this file against float64 (its bits stand for right ones above)."""
    offs = batch([300, 200, 2], [290, 200, 0], [2, 1], [300, 4000])
    run(offs, 4, 2, d, "bf16", "softmax")


def test_hook_refusals():
    plan = gd.PrefixPlan(*batch([5], [0], [1], [100]), 1, 64)
    for kw in (dict(limit_us=-1), dict(stall=-1), dict(stall=3)):
        with pytest.raises(gd.GdpaError) as e:
            plan.set_wait_test(**kw)
        assert e.value.status == 1
    assert np.all(np.array(plan.error_detail()) == 0)
