"""Failure path of the history cache's tensor-core kernels, without a GPU fault.

Every barrier wait is bounded.  The test hook shortens the limit to 20 ms and makes
the barriers of the first keys expect an arrival that never comes, so that waits for
them are never satisfied: the kernel must record a timeout, unwind (its copies and products in flight finish, TMEM
is freed) and return, check() must report GDPA_ERR_TIMEOUT with the place, and the
next call must be right.
"""

import ctypes
import time

import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from cache_util import Batch  # noqa: E402
from recommender_model_attention_gb300 import gdpa as raw  # noqa: E402

pytestmark = pytest.mark.gpu

TIMEOUT = 5   # GDPA_ERR_TIMEOUT
# wait sites of the warp-level kernel and of the tcgen05 kernel
MMA, TC = {1, 2}, set(range(61, 77))


def setup_module(_):
    gd.build()


@pytest.fixture(autouse=True)
def hook_off():
    yield
    gd.KVCache.set_wait_test()


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("new,hist,H,sites", [
    ([1], [0], 1, MMA), ([1] * 9, [3000] * 9, 8, MMA), ([2] * 5, [4000] * 5, 8, MMA), ([16, 16], [9000, 5], 2, MMA),
    ([40], [3], 1, TC), ([100, 90], [7000, 50], 1, TC), ([300, 400, 90], [2000, 9000, 10], 1, TC)])
def test_expired_wait_reports_timeout_and_cache_recovers(new, hist, H, sites, act, d, store):
    b = Batch(new, hist, H=H, Hkv=1, d=d, store=store, page=64).fill()
    o, lse = b.run(act)
    b.cache.check()
    gd.KVCache.set_wait_test(limit_us=20000, stall=1)
    t0 = time.time()
    b.run(act)
    detail = (ctypes.c_int32 * 4)()
    assert raw.lib().gdpa_cache_check(b.cache._ref, detail, torch.cuda.current_stream().cuda_stream) == TIMEOUT
    assert detail[0] == 1 and detail[1] in sites, list(detail)
    assert time.time() - t0 < 10.0
    # reported once; the next calls are right
    gd.KVCache.set_wait_test()
    b.cache.check()
    o2, lse2 = b.run(act)
    b.cache.check()
    assert torch.equal(o2, o) and (lse is None or torch.equal(lse2, lse))


def test_timeout_is_raised():
    b = Batch([1], [100]).fill()
    gd.KVCache.set_wait_test(limit_us=20000, stall=1)
    b.run()
    with pytest.raises(gd.GdpaError) as e:
        b.cache.check()
    assert e.value.status == TIMEOUT and "wait" in str(e.value)


def test_hook_refusals():
    for kw in (dict(limit_us=-1), dict(stall=-1), dict(stall=2)):
        with pytest.raises(gd.GdpaError) as e:
            gd.KVCache.set_wait_test(**kw)
        assert e.value.status == 1
