"""The history cache without a GPU: the oracle's own pins, and the refusals of
the C entry points (before any device is touched)."""

import ctypes
import math

import numpy as np
import pytest

import recommender_model_attention_gb300 as gd
from oracle import brute
from oracle import cache as orc
from recommender_model_attention_gb300 import gdpa as raw

OK, INVALID, UNSUPPORTED = 0, 1, 2


def setup_module(_):
    gd.build()


# ------------------------------------------------------------------ oracle

def test_codes_are_the_format_s():
    torch = pytest.importorskip("torch")
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(orc.e4m3_values(), codes)


def test_held_rounds_to_nearest_even():
    torch = pytest.importorskip("torch")
    x = torch.randn(300, 64, generator=torch.Generator().manual_seed(0)).double().numpy()
    x[:, 0] = 300.0        # fixes the exponent at 0
    x[0, 1:5] = [1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10]   # ties
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(orc.held(x, "e4m3"), want)
    assert list(want[0, 1:5]) == [1.0, 1.25, 0.0, 2.0 ** -8]
    # half a step at most: 2^-4 of a value, 2^-10 of the scale near zero
    y = np.ldexp(x, -7)
    assert np.all(np.abs(orc.held(y, "e4m3") - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -17))


def test_finite_rows_are_held_finite():
    top = 2.0 ** 128 - 2.0 ** 104                              # of float32
    x = np.array([[top, 248 * 2.0 ** 120, 247.9 * 2.0 ** 120, 1.0], [448 * 2.0 ** 119] * 4])
    want = [[240 * 2.0 ** 120] * 3 + [0.0], [448 * 2.0 ** 119] * 4]
    assert orc.held(x, "e4m3").tolist() == want
    assert (orc.held(-x, "e4m3") == -np.array(want)).all()


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7),
                                   (0.0, -126), (2.0 ** -140, -126), (3e38, 120)])
def test_exponents(top, e):
    assert orc.row_exponent(top) == e


def test_who_sees_what():
    # causal, window 2, one sink
    assert orc.sees(3, 2, "causal", 2, 1).astype(int).tolist() == [
        [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert orc.sees(2, 3, "history", 2, 0).astype(int).tolist() == [[0, 0, 1, 0, 0], [0, 0, 1, 0, 0]]
    # a root, two children, a grandchild of the first
    assert orc.sees(4, 1, "tree", 0, 0, [-1, 0, 0, 1]).astype(int).tolist() == [
        [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 1, 0, 1, 0], [1, 1, 1, 0, 1]]
    # positions along the path: the grandchild (3) is 2 from the root (1)
    assert orc.sees(4, 1, "tree", 2, 0, [-1, 0, 0, 1]).astype(int).tolist() == [
        [1, 1, 0, 0, 0], [0, 1, 1, 0, 0], [0, 1, 0, 1, 0], [0, 0, 1, 0, 1]]
    # a chain is the causal mask
    for w, s in ((0, 0), (3, 2)):
        assert np.array_equal(orc.sees(6, 4, "tree", w, s, [-1, 0, 1, 2, 3, 4]), orc.sees(6, 4, "causal", w, s))


def test_attention_is_softmax_over_the_events():
    rng = np.random.Generator(np.random.PCG64(0))
    q, k, v = rng.standard_normal((2, 2, 8)), rng.standard_normal((7, 1, 8)), rng.standard_normal((7, 1, 8))
    o, lse, _ = orc.attend([0, 2], [5], q, [k], [v], 0.3, "softmax")
    for h in range(2):
        x = 0.3 * k[:, 0] @ q[1, h]
        w = np.exp(x) / np.exp(x).sum()
        assert np.allclose(o[1, h], w @ v[:, 0], rtol=1e-13) and math.isclose(lse[1, h], math.log(np.exp(x).sum()))
        x = 0.3 * k[:6, 0] @ q[0, h]
        assert np.allclose(orc.attend([0, 2], [5], q, [k], [v], 0.3, "silu")[0][0, h], brute.act("silu", x) @ v[:6, 0])


# ---------------------------------------------------------------- refusals

A = 4096   # an address that is never followed


def cache(**kw):
    c = raw._CacheSpec(k=A, v=A, k_scale=A, v_scale=A, error=A, pages=4, page=64, heads=2, d=64, store=0)
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def where(table=A, off=A, starts=0, stride=4, width=4, B=2):
    return raw._cache_where(table, off, starts, stride, width, B)


def rows(x=A, token=128, head=64):
    return raw._cache_rows(x, token, head)


CACHES = [(dict(pages=-1), INVALID), (dict(heads=0), INVALID), (dict(d=0), INVALID), (dict(page=0), INVALID),
          (dict(store=3), INVALID), (dict(store=-1), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
          (dict(error=0), INVALID), (dict(error=A + 2), INVALID), (dict(k=A + 64), INVALID),
          (dict(store=2, k_scale=0), INVALID), (dict(store=2, v_scale=0), INVALID), (dict(store=2, v_scale=A + 1), INVALID),
          (dict(d=136), UNSUPPORTED), (dict(d=4), UNSUPPORTED), (dict(d=8, store=2), UNSUPPORTED),
          (dict(page=8), UNSUPPORTED), (dict(page=96), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
          (dict(heads=4097), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_caches_refused(kw, status):
    L, c = raw.lib(), cache(**kw)
    dt = 0
    assert L.gdpa_cache_write(ctypes.byref(c), dt, 5, rows(), rows(), where(), None) == status
    assert L.gdpa_cache_read(ctypes.byref(c), dt, 5, rows(), rows(), where(), None) == status
    attn = raw._cache_attn(0, 0, 0, 5, 1.0, 0)
    assert L.gdpa_cache_fwd(ctypes.byref(c), dt, 5, 4, rows(), A, None, where(), attn, A, 1 << 40, None) == status
    n = ctypes.c_int64()
    assert L.gdpa_cache_workspace(ctypes.byref(c), dt, 5, 4, 2, ctypes.byref(n)) == status
    assert L.gdpa_cache_check(ctypes.byref(c), (ctypes.c_int32 * 4)(), None) == status


def test_null_caches():
    L = raw.lib()
    assert L.gdpa_cache_write(None, 0, 5, rows(), rows(), where(), None) == INVALID
    assert L.gdpa_cache_bytes(None, None, None) == INVALID
    assert L.gdpa_cache_fwd(None, 0, 5, 4, rows(), A, None, where(), raw._cache_attn(0, 0, 0, 5, 1.0, 0), A, 1 << 40, None) == INVALID
    assert L.gdpa_cache_check(ctypes.byref(cache()), None, None) == INVALID


def test_sizes():
    L = raw.lib()
    a, b = ctypes.c_int64(), ctypes.c_int64()
    for store, row, scale in ((0, 128, 0), (1, 256, 0), (2, 64, 1)):
        c = cache(store=store, k=0, v=0, k_scale=0, v_scale=0, error=0, pages=70000)
        assert L.gdpa_cache_bytes(ctypes.byref(c), ctypes.byref(a), ctypes.byref(b)) == OK
        assert (a.value, b.value) == (70000 * 64 * 2 * row, 70000 * 64 * 2 * scale)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), INVALID), (dict(dt=1), INVALID), (dict(T=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=rows(0)), INVALID), (dict(v=rows(A + 1)), INVALID), (dict(w=None), INVALID), (dict(w=where(off=0)), INVALID),
    (dict(w=where(off=A + 2)), INVALID), (dict(w=where(table=0)), INVALID), (dict(w=where(table=A + 1)), INVALID),
    (dict(w=where(starts=A + 1)), INVALID), (dict(w=where(B=-1)), INVALID), (dict(w=where(width=-1)), INVALID),
    (dict(w=where(stride=-4)), INVALID),
    (dict(w=where(width=1 << 25)), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=0), OK), (dict(w=where(B=0, table=0)), OK),
    (dict(w=where(width=1 << 24)), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED)])
def test_rows_refused(kw, status):
    L, c = raw.lib(), cache()
    a = dict(dt=0, T=5, k=rows(), v=rows(), w=where())
    a.update(kw)
    for f in (L.gdpa_cache_write, L.gdpa_cache_read):
        assert f(ctypes.byref(c), a["dt"], a["T"], a["k"], a["v"], a["w"], None) == status


def test_reads_want_whole_pieces():
    L, c = raw.lib(), cache()
    for r in (rows(A + 2), rows(token=129), rows(head=65)):
        assert L.gdpa_cache_read(ctypes.byref(c), 0, 5, r, rows(), where(), None) == INVALID
        assert L.gdpa_cache_read(ctypes.byref(c), 0, 5, rows(), r, where(), None) == INVALID


def attn(mask=0, window=0, sinks=0, act=5, alpha=1.0, parents=0):
    return raw._cache_attn(mask, window, sinks, act, alpha, parents)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=3), INVALID), (dict(H=258), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(q=rows(0)), INVALID), (dict(q=rows(A + 1)), INVALID), (dict(o=0), INVALID),
    (dict(o=A + 8), INVALID), (dict(lse=A + 2), INVALID), (dict(lse=A, at=attn(act=2)), INVALID), (dict(at=None), INVALID),
    (dict(at=attn(mask=3)), INVALID), (dict(at=attn(mask=-1)), INVALID), (dict(at=attn(window=-1)), INVALID),
    (dict(at=attn(window=1, sinks=-1)), INVALID), (dict(at=attn(sinks=1)), INVALID), (dict(at=attn(act=6)), INVALID),
    (dict(at=attn(act=-1)), INVALID), (dict(at=attn(alpha=math.nan)), INVALID), (dict(at=attn(alpha=math.inf)), INVALID),
    (dict(at=attn(mask=2)), INVALID), (dict(at=attn(mask=2, parents=A + 1)), INVALID), (dict(w=where(off=0)), INVALID),
    (dict(T=1 << 30), UNSUPPORTED), (dict(T=0), OK), (dict(w=where(B=0, table=0)), OK)])
def test_attention_refused(kw, status):
    L, c = raw.lib(), cache()
    a = dict(dt=0, T=5, H=4, q=rows(), o=A, lse=None, w=where(), at=attn())
    a.update(kw)
    assert L.gdpa_cache_fwd(ctypes.byref(c), a["dt"], a["T"], a["H"], a["q"], a["o"], a["lse"], a["w"], a["at"], A,
                            1 << 40, None) == status


def test_workspace_refused():
    L, c, n = raw.lib(), cache(), ctypes.c_int64()
    for args in ((0, -1, 4, 2), (0, 5, 0, 2), (0, 5, 3, 2), (0, 5, 4, -1), (2, 5, 4, 2)):
        assert L.gdpa_cache_workspace(ctypes.byref(c), *args, ctypes.byref(n)) == INVALID
    assert L.gdpa_cache_workspace(ctypes.byref(c), 0, 5, 4, 2, None) == INVALID


@pytest.mark.parametrize("T,H", [(1 << 30, 4), (1 << 62, 4), ((1 << 63) - 1, 2), (5, 258), (1 << 29, 8), (1 << 24, 256)])
def test_workspace_of_sizes_that_attention_refuses(T, H):
    """... is refused the same way (products of such sizes leave 64 bits)."""
    L, c, n = raw.lib(), cache(), ctypes.c_int64(-7)
    assert L.gdpa_cache_workspace(ctypes.byref(c), 0, T, H, 2, ctypes.byref(n)) == UNSUPPORTED and n.value == -7
    assert L.gdpa_cache_fwd(ctypes.byref(c), 0, T, H, rows(), A, None, where(), attn(), A, 1 << 40, None) == UNSUPPORTED


def test_binding_refuses_host_memory():
    pytest.importorskip("torch")
    with pytest.raises(ValueError):
        gd.KVCache(1, 1, 64, device="cpu")


def test_wait_hook_refused():
    L = raw.lib()
    for args in ((-1, 0), (0, -1), (0, 2)):
        assert L.gdpa_cache_set_wait_test(*args) == INVALID
    assert L.gdpa_cache_set_wait_test(0, 0) == OK
