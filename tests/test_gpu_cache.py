"""The history cache on the GPU: rows written and read back, bit for bit."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from recommender_model_attention_gb300 import gdpa as raw  # noqa: E402
from cache_util import Batch, DT, dev, offsets, orc, ref  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(_):
    gd.build()


def same(a, b):
    assert np.array_equal(ref.to_f64(a), b, equal_nan=True)


@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 128), ("bf16", "bf16", 64), ("bf16", "bf16", 40),
                                           ("f32", "f32", 128), ("f32", "f32", 16), ("f32", "f32", 20),
                                           ("e4m3", "bf16", 128), ("e4m3", "bf16", 64), ("e4m3", "bf16", 48),
                                           ("e4m3", "f32", 128), ("e4m3", "f32", 16), ("e4m3", "f32", 112)])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_rows_come_back(store, dtype, d, page):
    b = Batch([3, 0, 1, 40, 17], [0, 5, 70, 33, 15], H=3, Hkv=3, d=d, store=store, dtype=dtype, page=page)
    b.fill()
    total = b.new + b.hist
    k, v = gd.gdpa_cache_read(b.cache, int(total.sum()), b.table, dev(offsets(total)), dtype=DT[dtype])
    b.cache.check()
    same(k, orc.held(ref.to_f64(b.k_all), store))
    same(v, orc.held(ref.to_f64(b.v_all), store))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_code_and_every_border_between_two(dtype):
    """Rows that hold each code, the middle of each two neighbours, and the
    nearest bf16 values on both sides, at scales from the least to the largest."""
    codes = orc.e4m3_values()
    mid = (codes[1:] + codes[:-1]) / 2
    near = np.concatenate([mid, mid * (1 - 2.0 ** -8), mid * (1 + 2.0 ** -7), codes])
    d, rows = 128, []
    for e in (-126, -125, -20, 0, 7, 100, 118):
        for i in range(0, len(near), 126):
            x = np.zeros(d)
            part = near[i:i + 126]
            x[:len(part)] = part
            x[127] = 448.0   # fixes the row's exponent
            rows.append(np.ldexp(np.where(np.arange(d) % 2 == 0, x, -x), e))
    # largest values on both sides of a step of the exponent
    for top in (448.0, 449.0, 447.0, 224.0, 2.0 ** -130, 2.0 ** -133, 0.0, 1.0, 3.0e38):
        x = np.full(d, top)
        x[1::2] = -top / 3
        rows.append(x)
    x = torch.from_numpy(np.array(rows)).to(DT[dtype])[:, None, :]
    n = x.shape[0]
    cache = gd.KVCache(2 * (n // 16 + 1), 1, d, page=16, store="e4m3")
    table = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda")[None]
    gd.gdpa_cache_write(cache, x.cuda(), -x.cuda(), table, dev([0, n]))
    k, v = gd.gdpa_cache_read(cache, n, table, dev([0, n]), dtype=torch.float32)
    want = orc.held(ref.to_f64(x), "e4m3")
    same(k, want)
    same(v, -want)
    # in bf16: the same values, rounded (exact but below its smallest normal number)
    k16, _ = gd.gdpa_cache_read(cache, n, table, dev([0, n]))
    same(k16, ref.to_f64(k.bfloat16()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_finite_rows_stay_finite(dtype):
    """Magnitudes whose nearest code stands for 2^128: the largest code below it."""
    top = torch.finfo(DT[dtype]).max
    rows = [top, 3.3e38, 248 * 2.0 ** 120, 247 * 2.0 ** 120, 232 * 2.0 ** 120, 448 * 2.0 ** 119]
    x = torch.zeros(2 * len(rows), 1, 64, dtype=torch.float64)
    for i, r in enumerate(rows):
        x[2 * i, 0, ::3] = r                       # beside zeros, and beside what rounds to less
        x[2 * i + 1, 0] = torch.linspace(-r, r, 64, dtype=torch.float64)
    x = x.to(DT[dtype])
    assert torch.isfinite(x).all()
    n = x.shape[0]
    cache = gd.KVCache(1, 1, 64, store="e4m3")
    args = (torch.zeros((1, 1), dtype=torch.int32, device="cuda"), dev([0, n]))
    gd.gdpa_cache_write(cache, x.cuda(), -x.cuda(), *args)
    for kind in (torch.float32, torch.bfloat16):
        k, v = gd.gdpa_cache_read(cache, n, *args, dtype=kind)
        want = orc.held(ref.to_f64(x), "e4m3")
        assert np.isfinite(want).all()
        same(k, want)
        same(v, -want)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_row_with_an_infinity_is_all_nan(bad):
    x = torch.randn(4, 2, 64)
    x[2, 1, 63] = bad
    cache = gd.KVCache(1, 2, 64, store="e4m3")
    args = (torch.zeros((1, 1), dtype=torch.int32, device="cuda"), dev([0, 4]))
    gd.gdpa_cache_write(cache, x.cuda(), x.cuda(), *args)
    k, v = gd.gdpa_cache_read(cache, 4, *args, dtype=torch.float32)
    for y in (k, v):
        nan = torch.isnan(y.cpu())
        assert nan[2, 1].all() and nan.sum() == 64
    # rows as they are keep it
    cache = gd.KVCache(1, 2, 64, store="f32")
    gd.gdpa_cache_write(cache, x.cuda(), x.cuda(), *args)
    same(gd.gdpa_cache_read(cache, 4, *args)[0], ref.to_f64(x))


@pytest.mark.parametrize("store,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strided_rows(store, dtype, shift):
    """K and V as parts of a packed projection, at any alignment of an element."""
    n, H, d = 37, 2, 64
    w = torch.randn(n, 3 * H * d + 8 + shift, dtype=torch.float32).to(DT[dtype]).cuda()
    k = w[:, shift:shift + H * d].view(n, H, d)
    v = w[:, shift + 2 * H * d:shift + 3 * H * d].unflatten(1, (d, H)).transpose(1, 2)   # columns not contiguous
    with pytest.raises(ValueError):
        gd.gdpa_cache_write(gd.KVCache(3, H, d, page=16, store=store), k, v, dev([[0, 1, 2]]), dev([0, n]))
    v = w[:, shift + H * d:shift + 2 * H * d].view(n, H, d).flip(1)
    v = torch.as_strided(w, (n, H, d), (w.stride(0), d, 1), shift + H * d)
    cache = gd.KVCache(3, H, d, page=16, store=store)
    gd.gdpa_cache_write(cache, k, v, dev([[2, 0, 1]]), dev([0, n]))
    out = torch.full((2, n, 2 * H, d), 7.0, dtype=DT[dtype], device="cuda")
    a, b = gd.gdpa_cache_read(cache, n, dev([[2, 0, 1]]), dev([0, n]), dtype=DT[dtype],
                              k_out=out[0, :, :H], v_out=out[1, :, H:])
    same(a, orc.held(ref.to_f64(k), store))
    same(b, orc.held(ref.to_f64(v), store))
    assert (out[0, :, H:] == 7).all() and (out[1, :, :H] == 7).all()


@pytest.mark.parametrize("store,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32")])
def test_strided_rows_with_heads_in_another_order(store, dtype):
    """K and V of strides of their own: V's heads lie further apart than its tokens."""
    n, H, d = 37, 2, 64
    k = torch.randn(n, H, d).to(DT[dtype]).cuda()
    v = torch.randn(H, n, d).to(DT[dtype]).cuda().transpose(0, 1)
    assert v.stride(0) < v.stride(1)
    cache = gd.KVCache(3, H, d, page=16, store=store)
    table, off = dev([[2, 0, 1]]), dev([0, n])
    gd.gdpa_cache_write(cache, k, v, table, off)
    out = torch.zeros(H, n, d, dtype=DT[dtype], device="cuda").transpose(0, 1)
    a, b = gd.gdpa_cache_read(cache, n, table, off, dtype=DT[dtype], v_out=out)
    same(a, orc.held(ref.to_f64(k), store))
    same(b, orc.held(ref.to_f64(v), store))
    assert b is out


def test_many_samples():
    """More samples than a block counts through."""
    n = 3000
    b = Batch([i % 3 for i in range(n)], [(i * 7) % 20 for i in range(n)], H=1, Hkv=1, d=64, store="bf16")
    b.fill()
    total = b.new + b.hist
    k, v = gd.gdpa_cache_read(b.cache, int(total.sum()), b.table, dev(offsets(total)))
    same(k, ref.to_f64(b.k_all))
    same(v, ref.to_f64(b.v_all))
    k, _ = gd.gdpa_cache_read(b.cache, int(b.new.sum()), b.table, b.off, b.starts)
    at = np.concatenate([f + h + np.arange(c) for f, h, c in zip(np.cumsum(total) - total, b.hist, b.new)]).astype(np.int64)
    same(k, ref.to_f64(b.k_all)[at])
    b.cache.check()


def test_rows_behind_the_last_sample_and_other_events_stay():
    cache = gd.KVCache(4, 1, 64, page=16)
    x = torch.randn(40, 1, 64).bfloat16().cuda()
    table = dev([[0, 1, 2, 3]])
    gd.gdpa_cache_write(cache, x, -x, table, dev([0, 40]))
    y = torch.randn(9, 1, 64).bfloat16().cuda()
    gd.gdpa_cache_write(cache, y, -y, table, dev([0, 3]), dev([14]))   # events 14, 15, 16; 6 rows are nobody's
    want = ref.to_f64(x).copy()
    want[14:17] = ref.to_f64(y)[:3]
    k, v = gd.gdpa_cache_read(cache, 40, table, dev([0, 40]))
    same(k, want)
    same(v, -want)
    out = torch.full((50, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    gd.gdpa_cache_read(cache, 50, table, dev([0, 40]), k_out=out)
    same(out[:40], want)
    assert (out[40:] == 3).all()


def test_nothing_to_do():
    cache = gd.KVCache(1, 1, 64)
    e = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    gd.gdpa_cache_write(cache, e, e, dev(np.zeros((0, 0))), dev([0]))
    k, v = gd.gdpa_cache_read(cache, 0, dev([[0]]), dev([0, 0]))
    assert k.shape == v.shape == (0, 1, 64)
    empty = gd.KVCache(0, 1, 64)
    gd.gdpa_cache_write(empty, e, e, dev([[0]]), dev([0, 0]))
    empty.check()


@pytest.mark.parametrize("table,off,starts,code", [([[5]], [0, 3], [0], 1), ([[-1]], [0, 3], [0], 1),
                                                   ([[0]], [0, 3], [14], 2), ([[0]], [0, 3], [-1], 2),
                                                   ([[0]], [0, 3], [2 ** 31 - 2], 2)])
def test_pages_and_events_outside_the_cache(table, off, starts, code):
    """Neither written nor read; recorded once, then cleared."""
    cache = gd.KVCache(2, 1, 64, page=16)
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    before = cache.k.clone()
    gd.gdpa_cache_write(cache, x, x, dev(table), dev(off), dev(starts))
    with pytest.raises(gd.GdpaError) as e:
        cache.check()
    assert e.value.status == 6
    cache.check()
    if code == 1:
        assert torch.equal(cache.k, before)
    k, _ = gd.gdpa_cache_read(cache, 3, dev(table), dev(off), dev(starts))
    with pytest.raises(gd.GdpaError):
        cache.check()
    inside = [0 <= starts[0] + i < 16 and code != 1 for i in range(3)]
    assert [bool((k[i] == 1).all()) for i in range(3)] == inside
    assert [bool((k[i] == 0).all()) for i in range(3)] == [not x for x in inside]


def detail(cache):
    """The record that gdpa_cache_check gives and clears: (status, what, sample, value)."""
    d = (ctypes.c_int32 * 4)()
    status = raw.lib().gdpa_cache_check(cache._ref, d, torch.cuda.current_stream().cuda_stream)
    if status:
        assert status == 6 and d[0] == 2
    return (status,) + tuple(d)[1:]


@pytest.mark.parametrize("table,start,what,values", [
    ([[0, 1], [2, 7]], 14, 1, {7}), ([[0, 1], [2, -3]], 14, 1, {-3}), ([[0, 1], [2, 1 << 30]], 14, 1, {1 << 30}),
    ([[0, 1], [2, 3]], 30, 2, {32}), ([[0, 1], [2, 3]], 100, 2, {100, 101, 102}), ([[0, 1], [2, 3]], -2, 2, {-2, -1}),
    ([[0, 1], [2, 3]], 2 ** 30, 2, {2 ** 30, 2 ** 30 + 1, 2 ** 30 + 2})])
def test_what_a_check_reports_of_rows(table, start, what, values):
    """Sample 1 of two is outside the cache: what, whose and which."""
    cache = gd.KVCache(4, 1, 64, page=16)
    x = torch.ones(5, 1, 64, dtype=torch.bfloat16, device="cuda")
    args = (dev(table), dev([0, 2, 5]), dev([3, start]))
    for call in (lambda: gd.gdpa_cache_write(cache, x, x, *args), lambda: gd.gdpa_cache_read(cache, 5, *args)):
        call()
        status, kind, sample, value = detail(cache)
        assert (status, kind, sample) == (6, what, 1) and value in values
        assert detail(cache) == (0, 0, 0, 0)


@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 64), ("f32", "f32", 64), ("bf16", "bf16", 48)])
@pytest.mark.parametrize("new", [1, 6, 80])
@pytest.mark.parametrize("table,start,what,value", [
    ([[0, 1, 2, 3, 4, 5, 6], [7, 99, 9, 10, 11, 12, 13]], 30, 1, 99), ([[0, 1, 2, 3, 4, 5, 6], [7, -8, 9, 10, 11, 12, 13]], 30, 1, -8),
    ([[0, 1, 2, 3, 4, 5, 6], [7, 8, 9, 10, 11, 12, 13]], 112, 2, 112), ([[0, 1, 2, 3, 4, 5, 6], [7, 8, 9, 10, 11, 12, 13]], -5, 3, -5)])
def test_what_a_check_reports_of_attention(table, start, what, value, new, store, dtype, d):
    cache = gd.KVCache(14, 1, d, page=16, store=store)
    q = torch.ones(2 * new, 1, d, dtype=DT[dtype], device="cuda")
    gd.gdpa_cache_softmax_fwd(cache, q, dev(table), dev([0, new, 2 * new]), dev([3, start]))
    assert detail(cache) == (6, what, 1, value)
    assert detail(cache) == (0, 0, 0, 0)


def test_offsets_that_pass_32_bits():
    """The last pages of a cache of more than 2^32 bytes a side."""
    pages, d = 9000, 128
    cache = gd.KVCache(pages, 8, d, page=256, store="bf16")   # 4.7 GB each
    assert cache.k.numel() > 2 ** 32
    x = torch.randn(300, 8, d).bfloat16().cuda()
    table, off = dev([[pages - 1, pages - 2]]), dev([0, 300])
    gd.gdpa_cache_write(cache, x, -x, table, off)
    k, v = gd.gdpa_cache_read(cache, 300, table, off)
    assert torch.equal(k, x) and torch.equal(v, -x)
    q = torch.randn(300, 8, d).bfloat16().cuda()
    o = gd.gdpa_cache_fwd(cache, q, table, off, act="identity")
    small = gd.KVCache(2, 8, d, page=256, store="bf16")
    gd.gdpa_cache_write(small, x, -x, dev([[0, 1]]), off)
    assert torch.equal(o, gd.gdpa_cache_fwd(small, q, dev([[0, 1]]), off, act="identity"))


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_rows_before_the_first_sample(store):
    """A part of a batch, by a part of its offsets: the others' rows stay as they are."""
    cache = gd.KVCache(4, 2, 64, page=16, store=store)
    x = torch.randn(20, 2, 64).bfloat16().cuda()
    gd.gdpa_cache_write(cache, x, x, dev([[0, 1]]), dev([0, 20]))
    want = [t.clone() for t in gd.gdpa_cache_read(cache, 20, dev([[0, 1]]), dev([0, 20]))]
    y = torch.randn(12, 2, 64).bfloat16().cuda()
    gd.gdpa_cache_write(cache, y, y, dev([[2], [0]]), dev([5, 9, 11]), dev([0, 14]))   # (events 9 .. 13 are whose rows 0 .. 4 would be)
    cache.check()
    k, v = gd.gdpa_cache_read(cache, 20, dev([[0, 1]]), dev([0, 20]))
    keep = [i for i in range(20) if i not in (14, 15)]
    assert torch.equal(k[keep], want[0][keep]) and torch.equal(v[keep], want[1][keep])
    out = torch.full((12, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k, _ = gd.gdpa_cache_read(cache, 12, dev([[2], [0]]), dev([5, 9, 11]), dev([0, 14]), k_out=out)
    assert (k[:5] == 7).all() and (k[11:] == 7).all()
    if store == "bf16":
        assert torch.equal(k[5:11], y[5:11])


def test_a_wait_that_ran_out_is_a_timeout():
    cache = gd.KVCache(1, 1, 64)
    cache.error.copy_(dev([1, 71, 3, 0]))
    with pytest.raises(gd.GdpaError) as e:
        cache.check()
    assert e.value.status == 5 and "wait 71" in str(e.value)
    cache.check()


def test_refusals():
    with pytest.raises(KeyError):
        gd.KVCache(1, 1, 64, store="int8")
    for kw in (dict(d=136), dict(d=60), dict(page=8), dict(page=48), dict(page=2048), dict(heads=5000)):
        with pytest.raises(gd.GdpaError) as e:
            gd.KVCache(1, kw.pop("heads", 1), kw.pop("d", 64), **kw)
        assert e.value.status == 2
    with pytest.raises(gd.GdpaError):
        gd.KVCache(1, 1, 72, store="e4m3")   # 72 bytes a row
    for pages, heads, d in ((-1, 1, 64), (1, 0, 64), (1, 1, 0)):
        with pytest.raises(gd.GdpaError) as e:
            gd.KVCache(pages, heads, d)
        assert e.value.status == 1
    c = gd.KVCache(2, 2, 64)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    t, off = dev([[0]]), dev([0, 5])
    bad = [(x.float(), x, t, off), (x, x.float(), t, off), (x[:, :1], x, t, off), (x, x[:4], t, off),
           (x, x, t, dev([0, 2, 5])), (x, x, t.long(), off), (x, x, t[0], off), (x, x, t, off.cpu()),
           (x.cpu(), x, t, off), (x, x, t, off, dev([0, 1])), (x, x, t, off, dev([0]).long()), (x, x, t, None)]
    for args in bad:
        with pytest.raises((ValueError, TypeError)):
            gd.gdpa_cache_write(c, *args)
    with pytest.raises(TypeError):
        gd.gdpa_cache_read(c, 5, t, off, dtype=torch.float32)
    with pytest.raises(ValueError):
        gd.gdpa_cache_read(c, 5, t, off, k_out=x[:4])
    with pytest.raises(ValueError):
        gd.gdpa_cache_read(c, 5, t, off, k_out=x[:1].expand(5, 2, 64))
    wide = torch.zeros(5, 2, 65, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gd.GdpaError) as e:   # rows that are not in 16-byte pieces
        gd.gdpa_cache_read(c, 5, t, off, k_out=wide[:, :, :64])
    assert e.value.status == 1
