"""Attention over the history cache on the GPU against the float64 oracle.
Bounds: cache_util.check_o."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from recommender_model_attention_gb300 import gdpa as raw  # noqa: E402
from cache_util import Batch, check_lse, check_o, dev, offsets, orc, ref  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16", 128), ("bf16", "bf16", 64), ("e4m3", "bf16", 128), ("e4m3", "bf16", 64),
         ("f32", "f32", 32), ("e4m3", "f32", 64), ("bf16", "bf16", 40), ("e4m3", "bf16", 48), ("f32", "f32", 128)]
SHAPES = {
    "one event": ([1], [0]),
    "one row": ([1], [100]),
    "single rows": ([1] * 9, [0, 1, 15, 16, 17, 63, 64, 65, 200]),
    "ragged": ([3, 0, 1, 20, 2, 9], [0, 5, 300, 33, 1, 0]),
    "group edges": ([16, 15, 17, 1], [16, 17, 15, 47]),
    "many rows": ([70, 130], [40, 3]),
}


def setup_module(_):
    gd.build()


def tree(new, seed=0):
    """Parents of drafted rows: chains, wide trees and several roots."""
    rng = np.random.Generator(np.random.PCG64(seed))
    return [int(rng.integers(max(-1, i - 6), i)) for n in new for i in range(n)]


@pytest.mark.parametrize("store,dtype,d", KINDS)
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_shapes(shape, act, store, dtype, d):
    b = Batch(*SHAPES[shape], H=4, Hkv=2, d=d, store=store, dtype=dtype).fill()
    b.check(act)


@pytest.mark.parametrize("store,dtype,d", KINDS[:6])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 0), (20, 1), (20, 5), (33, 40), (1, 16), (1000, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("mask", ["causal", "history", "tree"])
def test_windows_and_sinks(store, dtype, d, window, sinks, mask):
    new = [1, 30, 5, 0, 18]
    b = Batch(new, [150, 70, 0, 40, 19], d=d, store=store, dtype=dtype,
              parents=tree(new) if mask == "tree" else None).fill()
    b.check("softmax", mask=mask, window=window, sinks=sinks)
    b.check("gelu_tanh", mask=mask, window=window, sinks=sinks)


@pytest.mark.parametrize("store,dtype,d", KINDS[:6])
@pytest.mark.parametrize("act", ["softmax", "gelu_erf"])
def test_trees(store, dtype, d, act):
    new = [24, 1, 64, 0, 7, 100]
    for seed, hist in enumerate(([130, 0, 17, 9, 0, 40], [0] * 6)):
        b = Batch(new, hist, H=4, Hkv=1, d=d, store=store, dtype=dtype, parents=tree(new, seed)).fill()
        b.check(act, mask="tree")


def test_special_trees():
    n = 40
    chain = [i - 1 for i in range(n)]
    b = Batch([n], [37], parents=chain).fill()
    o, lse = b.check(mask="tree")
    c, clse = b.run(mask="tree"), None
    b.parents, b.parents_host = None, None
    o2, lse2 = b.run(mask="causal")     # a chain is the causal mask
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    Batch([n], [37], parents=[-1] * n).fill().check(mask="tree")              # no two rows see each other
    Batch([n], [37], parents=[-1] + [0] * (n - 1)).fill().check(mask="tree")  # a star
    # what is no row before the own one is no parent
    odd = [0, 5, 1, 3, -7, 2 ** 31 - 1, 2, -2 ** 31]
    Batch([8], [3], parents=odd).fill().check(mask="tree")


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 8), (8, 1), (6, 2), (40, 1), (128, 1), (24, 8)])
@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 128), ("e4m3", "bf16", 64), ("f32", "f32", 16)])
def test_shared_key_heads(H, Hkv, store, dtype, d):
    b = Batch([1, 3, 0, 2], [40, 7, 3, 130], H=H, Hkv=Hkv, d=d, store=store, dtype=dtype).fill()
    b.check()
    b.check("gelu_tanh")


@pytest.mark.parametrize("act", ["softmax", "gelu_erf", "gelu_tanh", "silu", "gelu_taylor6", "identity"])
@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 128), ("e4m3", "bf16", 128), ("e4m3", "f32", 48)])
def test_activations(act, store, dtype, d):
    b = Batch([5, 1, 9], [100, 30, 0], d=d, store=store, dtype=dtype, gain=0.5).fill()   # the polynomial's range
    b.check(act)
    b.check(act, alpha=0.0)
    b.check(act, alpha=-0.05)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_pages(page, store):
    Batch([3, 1, 20], [100, 1500, 15], page=page, store=store, extra_width=2).fill().check()


@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 128), ("e4m3", "bf16", 128), ("f32", "f32", 32)])
def test_long_histories_are_split(store, dtype, d):
    """One user's events over all CTAs, beside short ones; rows of several tiles."""
    b = Batch([1, 2, 1], [30000, 11, 4000], H=2, Hkv=1, d=d, store=store, dtype=dtype, page=64).fill()
    b.check()
    b.check("silu", alpha=0.01)
    b = Batch([40, 1], [9000, 100], H=2, Hkv=1, d=d, store=store, dtype=dtype, page=64).fill()
    b.check()


def test_many_samples():
    n = 1500
    new = [(i * 5) % 3 for i in range(n)]
    Batch(new, [(i * 11) % 40 for i in range(n)], H=1, Hkv=1, d=64).fill().check()
    # few samples with rows between many without
    new = [0] * n
    new[3], new[700], new[1499] = 2, 1, 3
    Batch(new, [20] * n, H=1, Hkv=1, d=64, store="e4m3").fill().check()


@pytest.mark.parametrize("store,dtype,d", KINDS[:6])
def test_rows_that_see_nothing(store, dtype, d):
    b = Batch([2, 1, 3], [0, 50, 0], d=d, store=store, dtype=dtype).fill()
    o, lse = b.check(mask="history")
    assert (o[:2] == 0).all() and (o[3:] == 0).all() and torch.isinf(lse[:2]).all()
    assert (b.check("silu", mask="history")[0][:2] == 0).all()


@pytest.mark.parametrize("store,dtype,d", KINDS[:6])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("act", ["softmax", "silu"])
def test_hidden_events_may_hold_anything(store, dtype, d, bad, act):
    """Rows hidden by the window, by the causal order or by the tree hold NaN or
    infinities: rows that do not see them are as without them."""
    new, hist = [20, 3], [40, 33]
    parents = tree(new, 3)
    for mask in ("causal", "tree", "history"):
        b = Batch(new, hist, d=d, store=store, dtype=dtype, parents=parents if mask == "tree" else None)
        clean, clean_lse = b.fill().run(act, mask=mask, window=9, sinks=2)
        kw = dict(mask=mask, window=9, sinks=2)
        see = [orc.sees(n, h, mask, 9, 2, parents[:20] if i == 0 else parents[20:]) for i, (n, h) in enumerate(zip(new, hist))]
        victim = 43 if mask != "history" else 36      # a new row of sample 0; an event that its window hides later
        for x in (b.k_all, b.v_all):
            x[victim] = bad
            x[60 + 5] = bad                           # an event of sample 1 that nobody sees
        o, lse = b.fill().run(act, **kw)
        assert not see[1][:, 5].any()
        hit = np.concatenate([see[0][:, victim], np.zeros(3, dtype=bool)])
        assert hit.any() and not hit.all() or mask == "history"
        ok = torch.from_numpy(~hit).cuda()
        assert torch.equal(o[ok], clean[ok])
        assert torch.isnan(o[~ok]).all() or act != "softmax"
        if lse is not None:
            assert torch.equal(lse[ok], clean_lse[ok])


@pytest.mark.parametrize("act", ["softmax", "silu"])
def test_value_rows_of_very_different_sizes(act):
    """8-bit rows whose powers of two span 2^-40 .. 2^40: to each output's own
    terms, wherever in the history the large ones lie."""
    for seed, order in enumerate((1, -1, 0)):
        b = Batch([1, 2], [600, 333], store="e4m3", seed=seed, gain=2.0)
        n = b.v_all.shape[0]
        e = np.linspace(-40, 40, n).round()[::order or 1]
        if order == 0:
            e = np.random.Generator(np.random.PCG64(5)).permutation(e)
        b.v_all = b.v_all * torch.from_numpy(np.ldexp(1.0, e.astype(int))).to(torch.bfloat16)[:, None, None]
        b.fill().check(act)


@pytest.mark.parametrize("store,dtype,d", KINDS[:5])
def test_large_scores(store, dtype, d):
    """Scores of hundreds that rise along the history: the reference moves at
    most groups, and at the end one event has nearly all the weight."""
    b = Batch([2, 1], [700, 90], d=d, store=store, dtype=dtype)
    n = b.k_all.shape[0]
    b.k_all = (b.k_all.float() * torch.linspace(0.1, 30, n)[:, None, None]).to(b.k_all.dtype)
    o, lse = b.fill().run()
    want, wlse, size = b.want(d ** -0.5, "softmax")
    err = np.abs(ref.to_f64(o) - want)
    # a score of up to X = 30 * 1.5 * sqrt(d) is summed in float32 from d terms of
    # together at most X: off by d 2^-24 X at most, 128 * 2^-24 * 510 = 3.9e-3, which
    # a weight is off by relatively
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 3.9e-3) * size[0] + 1e-30)
    assert np.max(np.abs(ref.to_f64(lse) - wlse)) <= 2 * 3.9e-3


def flat_tail(new, H, d, nats, events, spread, at, store, dtype=None):
    """One event `nats` above a tail of scores N(0, spread), new * H rows."""
    b = Batch([new], [events], H=H, Hkv=1, d=d, store=store, dtype=dtype, page=64)
    g = torch.Generator().manual_seed(at + 1)
    u = torch.randn((d,), generator=g).bfloat16().float()
    b.q = (u * (1 + torch.arange(new * H) / 256.0)[:, None]).view(new, H, d).to(b.dt).cuda()
    unit = d ** 0.5 / u.square().sum()           # of a key along u whose score is 1
    n = events + new
    b.k_all = (spread * d ** 0.5 / u.norm() * torch.randn((n, 1, d), generator=g)).to(b.dt)
    b.k_all[at, 0] = (u * unit * nats).to(b.dt)
    b.v_all = (2.5 + 2.5 * torch.rand((n, 1, d), generator=g)).to(b.dt)
    b.v_all[:, :, 7] = 5.0                       # fixes the rows' powers of two
    b.v_all[at, :, :4] = 0.0
    return b


def run_shared(b, many):
    """The batch's one sample, many times on the same pages (so that most of a
    history is one CTA's), against what it should give once."""
    new, events = int(b.new[0]), int(b.hist[0])
    b.fill()
    want, wlse, size = b.want(b.d ** -0.5, "softmax", mask="history")
    o, lse = gd.gdpa_cache_softmax_fwd(b.cache, b.q.repeat(many, 1, 1), b.table.expand(many, -1),
                                       dev(new * np.arange(many + 1)), dev([events] * many), mask="history")
    b.cache.check()
    rep = lambda x: np.tile(x, (many,) + (1,) * (x.ndim - 1))  # noqa: E731
    check_o(o, rep(want), [rep(x) for x in size], "softmax", b)
    check_lse(lse, rep(wlse))


@pytest.mark.parametrize("store,dtype,d,new,H", [("bf16", "bf16", 128, 1, 1), ("bf16", "bf16", 64, 2, 8), ("bf16", "bf16", 128, 4, 8),
                                                 ("bf16", "bf16", 64, 9, 8), ("bf16", "bf16", 48, 1, 1), ("f32", "f32", 128, 1, 1),
                                                 ("f32", "f32", 32, 1, 4), ("e4m3", "f32", 64, 1, 1), ("f32", "f32", 64, 2, 8)])
def test_sums_of_many_equal_weights(store, dtype, d, new, H):
    """Thousands of equal weights beside one of e^9: their sum is not to drift with
    the rounding of each (one after the other, up to 2^-24 of the sum each)."""
    run_shared(flat_tail(new, H, d, 9, 16000, 0.0, 0, store, dtype), 600)


@pytest.mark.parametrize("nats,events,spread", [(9, 16000, 0.0), (11.5, 16000, 0.0), (14, 16000, 0.0), (13, 16000, 1.0),
                                                (30, 60000, 0.0)])
@pytest.mark.parametrize("new,H", [(1, 1), (1, 8), (2, 8), (4, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_one_event_far_above_a_long_flat_tail(d, new, H, nats, events, spread):
    """What `sinks` are for: the tail keeps its share, also in columns that the
    event above it does not fill.  (30 nats: the 31 events that are weighed beside it
    may be lost, 31 / 60000 of the tail, 2^-10.9 of such a column's value: less than
    the 2^-11 + 2^-12 of the terms that the bound has for rounded weights.)"""
    for at in (0, events // 2):
        run_shared(flat_tail(new, H, d, nats, events, spread, at, "e4m3"), 600)


MANY = ([70, 130, 0, 33, 1], [40, 3, 20, 300, 0])   # more than 32 rows a sample on average
TC = [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64)]


@pytest.mark.parametrize("store,d", TC)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 5), (64, 130), (150, 0), (2 ** 31 - 1, 1)])
@pytest.mark.parametrize("mask", ["causal", "history", "tree"])
def test_many_rows_windows_and_sinks(store, d, window, sinks, mask):
    b = Batch(*MANY, d=d, store=store, parents=tree(MANY[0]) if mask == "tree" else None).fill()
    b.check("softmax", mask=mask, window=window, sinks=sinks)
    b.check("silu", mask=mask, window=window, sinks=sinks)


@pytest.mark.parametrize("store,d", TC)
@pytest.mark.parametrize("act", ["softmax", "gelu_erf", "gelu_tanh", "silu", "gelu_taylor6", "identity"])
def test_many_rows_activations(store, d, act):
    b = Batch(*MANY, H=4, Hkv=2, d=d, store=store, gain=0.5, page=64).fill()
    b.check(act)
    b.check(act, alpha=0.0)
    b.check(act, alpha=-0.05)
    b.check(act, mask="history")


@pytest.mark.parametrize("store,d", TC)
@pytest.mark.parametrize("H,Hkv", [(3, 1), (128, 1), (10, 2)])
def test_many_rows_shared_key_heads(store, d, H, Hkv):
    """Tiles of one, two and more row blocks, and of tokens cut between them."""
    Batch([2, 45, 7], [300, 130, 1], H=H, Hkv=Hkv, d=d, store=store).fill().check()


@pytest.mark.parametrize("store,d", TC)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_many_rows_hidden_events_may_hold_anything(store, d, bad):
    new, hist = [90, 40], [70, 33]
    parents = tree(new, 3)
    for mask, act in (("causal", "softmax"), ("tree", "softmax"), ("causal", "silu")):
        b = Batch(new, hist, d=d, store=store, parents=parents if mask == "tree" else None)
        kw = dict(mask=mask, window=30, sinks=2)
        clean, clean_lse = b.fill().run(act, **kw)
        see = orc.sees(90, 70, mask, 30, 2, parents[:90])
        b.k_all[100], b.v_all[100] = bad, bad       # new row 30 of sample 0
        b.v_all[120, 1, 5] = bad                    # one value of new row 50
        o, lse = b.fill().run(act, **kw)
        hit = np.concatenate([see[:, 100], np.zeros(40, dtype=bool)])
        part = np.concatenate([see[:, 120], np.zeros(40, dtype=bool)])
        assert hit.any() and part.any() and not (hit | part).all()
        ok = torch.from_numpy(~(hit | part)).cuda()
        assert torch.equal(o[ok], clean[ok])
        assert not torch.isfinite(o[torch.from_numpy(hit).cuda()]).any() or act != "softmax"
        only = torch.from_numpy(part & ~hit).cuda()
        assert not torch.isfinite(o[only][:, 1, 5]).any()
        if store == "bf16":                         # (8-bit: the whole row of that head is NaN)
            keep = torch.ones(d, dtype=torch.bool, device="cuda")
            keep[5] = False
            assert torch.equal(o[only][:, 0], clean[only][:, 0]) and torch.equal(o[only][:, 1][:, keep], clean[only][:, 1][:, keep])
        if lse is not None:
            assert torch.equal(lse[ok], clean_lse[ok])


@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 128), ("bf16", "bf16", 64), ("f32", "f32", 64), ("bf16", "bf16", 48),
                                           ("e4m3", "bf16", 128), ("e4m3", "f32", 64)])
@pytest.mark.parametrize("new,H", [([1, 1], 2), ([3, 2], 2), ([9, 12], 2), ([20, 30], 2), ([40, 100], 2), ([100, 100], 2), ([300, 9], 2)])
@pytest.mark.parametrize("act", ["softmax", "silu"])
def test_visible_infinities_and_nans_are_seen(act, new, H, store, dtype, d):
    """Wherever such an event lies, in blocks that all rows see or some, the rows that
    see it have no finite number in its column, and all else is as without it, also
    where the event's weight is tiny (its key far below the others)."""
    hist = [700, 300]
    for far in (False, True) if act == "softmax" else (False,):
        for event in (0, 130, 255, 640, 699, hist[0] + new[0] // 2):
            b = Batch(new, hist, H=H, Hkv=2, d=d, store=store, dtype=dtype, gain=0.5)
            if far:                                  # all but the 128 around it 150 nats above
                b.q[:new[0]] = 1.0
                b.k_all[:hist[0] + new[0]] = 0.5
                at = event - event % 128
                b.k_all[at:min(at + 128, hist[0] + new[0])] = 0.5 - 150 * d ** -0.5
            clean, lse = b.fill().run(act)
            hit = np.concatenate([event <= hist[0] + np.arange(new[0]), np.zeros(new[1], dtype=bool)])
            on = torch.from_numpy(hit).cuda()
            same = torch.ones(clean.shape, dtype=torch.bool, device="cuda")
            same[on, 1] = store != "e4m3"            # (8-bit: the whole row of that head is NaN)
            same[on, 1, 5] = False
            for bad in (float("inf"), -float("inf"), float("nan")):
                b.v_all[event, 1, 5] = bad
                o, l2 = b.fill().run(act)
                assert not torch.isfinite(o[on][:, 1, 5]).any(), (bad, event, far)
                assert torch.equal(o[same], clean[same]), (bad, event, far)
                if lse is not None:
                    assert torch.equal(l2, lse)


@pytest.mark.parametrize("store,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64)])
@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("every", [1, 5, 7])
def test_bad_events_of_some_samples_among_many(every, act, store, d):
    """Several samples a CTA one after the other: those with a NaN in a block that
    some of their rows do not see, and those without."""
    n = 1600
    new = [40 + i % 3 for i in range(n)]
    b = Batch(new, [(i * 37) % 150 for i in range(n)], H=1, Hkv=1, d=d, store=store).fill()
    clean, lse = b.run(act)
    first = np.cumsum(b.new + b.hist) - (b.new + b.hist)
    hit = np.zeros(sum(new), dtype=bool)
    for s in range(0, n, every):
        b.v_all[first[s] + b.hist[s] + 20] = float("nan")   # new row 20
        hit[b.off_host[s] + 20:b.off_host[s + 1]] = True
    o, l2 = b.fill().run(act)
    hit = torch.from_numpy(hit).cuda()
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])
    assert lse is None or torch.equal(l2, lse)


def poke(b, event, scale, code):
    """The values of an event of sample 0 in an 8-bit cache's memory: `code` in
    every column and a scale byte (a page that was never written, or another's)."""
    page, e = int(b.table_host[0, event // b.page]), event % b.page
    block = b.cache.v.view(-1)[:b.cache.pages * b.Hkv * b.page * b.d].view(b.cache.pages, b.Hkv, b.page, b.d)
    block[page, :, e] = code      # (a row's bytes lie together, in some order)
    b.cache.v_scale.view(-1)[:b.cache.pages * b.Hkv * b.page].view(b.cache.pages, b.Hkv, b.page)[page, :, e] = scale


@pytest.mark.parametrize("new", [[90, 40], [300, 10], [3, 2], [1, 1], [20, 12]])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (64, "f32")])
@pytest.mark.parametrize("act", ["softmax", "silu"])
def test_hidden_values_of_any_scale(act, d, dtype, new):
    """Codes and scales whose product no float32 holds, in events that some rows do
    not see: those rows are as without them."""
    hist = [70, 33]
    b = Batch(new, hist, d=d, store="e4m3", dtype=dtype)
    kw = dict(window=30, sinks=2)
    clean, clean_lse = b.fill().run(act, **kw)
    see = orc.sees(new[0], hist[0], "causal", 30, 2)
    for scale in (246, 247, 248, 251, 254, 255):
        for code in (0x7e, 0xfe, 0x78, 0x08, 0x00):
            for victim in {69, hist[0] + new[0] // 3, 20}:
                b.fill()
                poke(b, victim, scale, code)
                o, lse = b.run(act, **kw)
                hit = np.concatenate([see[:, victim], np.zeros(new[1], dtype=bool)])
                ok = torch.from_numpy(~hit).cuda()
                assert torch.equal(o[ok], clean[ok]), (scale, code, victim)
                if lse is not None:
                    assert torch.equal(lse, clean_lse)
                if scale == 255 and hit.any():      # (the byte of rows of NaNs)
                    assert not torch.isfinite(o[~ok]).any()
                if code == 0 and scale == 246:
                    assert torch.isfinite(o).all()


@pytest.mark.parametrize("store,d", TC)
def test_many_rows_pages_outside_the_cache(store, d):
    """Missing pages are as hidden events, also inside blocks that every row sees."""
    b = Batch([64, 50], [500, 30], d=d, store=store).fill()
    good, _ = b.run()
    b.table_host[0, 3] = 1 << 20     # events 48 .. 63 of sample 0
    b.table_host[0, 33] = -1         # events 528 .. 543, new rows 28 .. 43
    b.table = dev(b.table_host)
    o, _ = b.run()
    with pytest.raises(gd.GdpaError):
        b.cache.check()
    assert torch.equal(o[64:], good[64:])
    keep = np.array([j for j in range(564) if not 48 <= j < 64 and not 528 <= j < 544])
    k, v = (orc.held(ref.to_f64(x), store)[:564][keep] for x in (b.k_all, b.v_all))
    for i in (0, 30, 63):
        see = keep <= 500 + i
        want, _, size = orc.attend([0, 1], [see.sum() - 1], ref.to_f64(b.q[i:i + 1]), [k[see]], [v[see]], d ** -0.5, "softmax")
        check_o(o[i:i + 1], want, size, "softmax", b)


def test_many_rows_large_scores_and_sizes():
    """References that move along the history, and 8-bit rows of sizes 2^-40 .. 2^40."""
    for store in ("bf16", "e4m3"):
        b = Batch([40, 60], [700, 90], store=store)
        n = b.k_all.shape[0]
        b.k_all = (b.k_all.float() * torch.linspace(0.1, 30, n)[:, None, None]).to(b.k_all.dtype)
        o, lse = b.fill().run()
        want, wlse, size = b.want(128 ** -0.5, "softmax")
        # as test_large_scores
        assert np.all(np.abs(ref.to_f64(o) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 3.9e-3) * size[0] + 1e-30)
        assert np.max(np.abs(ref.to_f64(lse) - wlse)) <= 2 * 3.9e-3
        b = Batch([40, 60], [300, 90], store=store, seed=2)
        n = b.v_all.shape[0]
        e = np.random.Generator(np.random.PCG64(5)).permutation(np.linspace(-40, 40, n).round())
        b.v_all = b.v_all * torch.from_numpy(np.ldexp(1.0, e.astype(int))).to(torch.bfloat16)[:, None, None]
        b.fill().check()
        b.check("silu")


@pytest.mark.parametrize("new,H,store,dtype,d", [([1, 1], 2, "f32", "f32", 64), ([9, 7], 2, "f32", "f32", 64), ([1, 1], 2, "e4m3", "bf16", 48)]
                         + [(n, 2, s, "bf16", d) for n in ([3, 2], [12, 20], [20, 40], [90, 100], [200, 90]) for s, d in TC])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_queries_with_infinities_and_nans(new, H, store, dtype, d, bad):
    """Their rows are NaN, and theirs alone."""
    b = Batch(new, [40, 200], H=H, Hkv=2, d=d, store=store, dtype=dtype).fill()
    good, lse = b.run()
    b.q[1, 0, 3] = bad
    o, l2 = b.run()
    assert torch.isnan(o[1, 0]).all() and torch.isnan(l2[1, 0])
    same = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
    same[1, 0] = False
    assert torch.equal(o[same], good[same]) and torch.equal(l2[same], lse[same])


def test_part_of_a_batch():
    """Offsets that start behind the first row: others' outputs stay as they are."""
    for store, d, dtype in (("bf16", 128, None), ("f32", 64, None), ("e4m3", 48, "bf16")):
        for new in ([1, 2, 1, 1], [9, 3, 7, 20], [60, 40, 90, 33]):
            b = Batch(new, [50, 7, 90, 300], d=d, store=store, dtype=dtype).fill()
            want, _ = b.run()
            o = torch.full_like(b.q, 7.0)
            gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table[1:3], b.off[1:4].clone(), b.starts[1:3].clone(), o=o)
            lo, hi = int(b.off_host[1]), int(b.off_host[3])
            assert (o[:lo] == 7).all() and (o[hi:] == 7).all()
            assert torch.allclose(o[lo:hi].float(), want[lo:hi].float(), rtol=2.0 ** -6, atol=2.0 ** -7)


def test_two_graphs_and_two_streams_at_once():
    """Two captured calls and one of another stream, of three batches, under way
    side by side: each has its own workspace."""
    sizes = ([[1] * 8, [5000] * 8], [[40] * 6, [900] * 6], [[6] * 7, [3000] * 7])
    batches = [Batch(n, h, H=4, Hkv=2, d=128, store="e4m3", page=64, seed=i).fill() for i, (n, h) in enumerate(sizes)]
    want = [b.run() for b in batches]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in batches[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    eager = []
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        b = batches[2]
        eager.append(gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table, b.off, b.starts, stream=streams[2]))
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs + eager, want[:2] + [want[2]] * 20):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_long_shares_of_many_tiles(store):
    """Shares of more than 512 groups, which take what another began of an item last."""
    rng = np.random.Generator(np.random.PCG64(3))
    b = Batch([512, 700, 300, 512, 640, 90, 512, 800], rng.integers(8000, 11000, 8), H=8, Hkv=2, store=store, page=64).fill()
    o, lse = b.run()
    b.cache.check()
    for s, (k, v) in enumerate(zip(b.split(b.k_all), b.split(b.v_all))):
        k, v = (orc.held(ref.to_f64(x), store) for x in (k, v))
        for i in sorted({0, 63, int(b.new[s]) // 2, int(b.new[s]) - 1} & set(range(int(b.new[s])))):
            t, see = int(b.off_host[s]) + i, int(b.hist[s]) + i + 1
            want, wlse, size = orc.attend([0, 1], [see - 1], ref.to_f64(b.q[t:t + 1]), [k[:see]], [v[:see]], 128 ** -0.5, "softmax")
            check_o(o[t:t + 1], want, size, "softmax", b)
            check_lse(lse[t:t + 1], wlse)


def test_outputs_over_the_queries():
    for new, H, store, dtype, d in (([1, 3], 8, "e4m3", "bf16", 128), ([70, 90], 2, "bf16", "bf16", 64), ([1, 2], 1, "f32", "f32", 64)):
        b = Batch(new, [5000, 300], H=H, Hkv=1, d=d, store=store, dtype=dtype, page=64).fill()
        want, lse = b.run()
        q = b.q.clone()
        o, l2 = gd.gdpa_cache_softmax_fwd(b.cache, q, b.table, b.off, b.starts, o=q)
        assert torch.equal(o, want) and torch.equal(l2, lse)


def test_samples_that_share_pages():
    """One history for all samples (a table that is expanded)."""
    b = Batch([1], [400], H=4, Hkv=2, d=64, store="e4m3").fill()
    q = torch.randn(6, 4, 64, device="cuda").bfloat16()
    many = gd.gdpa_cache_softmax_fwd(b.cache, q, b.table.expand(6, -1), dev(np.arange(7)), dev([400] * 6), mask="history")
    one = gd.gdpa_cache_softmax_fwd(b.cache, q, b.table, dev([0, 6]), dev([400]), mask="history")
    for x, y in zip(many, one):   # other tiles: other orders of the sums
        assert torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=2.0 ** -8)


def test_strided_queries():
    b = Batch([5, 3], [50, 20], H=4, Hkv=2, d=64).fill()
    want, lse = b.run()
    for shift in (0, 1, 8):
        w = torch.zeros(8, 9 * 64 + shift, dtype=torch.bfloat16, device="cuda")
        q = torch.as_strided(w, (8, 4, 64), (w.stride(0), 128, 1), shift)
        q.copy_(b.q)
        o, l2 = gd.gdpa_cache_softmax_fwd(b.cache, q, b.table, b.off, b.starts)
        assert torch.equal(o, want) and torch.equal(l2, lse)


@pytest.mark.parametrize("store,dtype,d", [("bf16", "bf16", 128), ("e4m3", "bf16", 128), ("e4m3", "bf16", 64), ("e4m3", "f32", 64), ("f32", "f32", 64)])
@pytest.mark.parametrize("new", [[1, 1], [9, 12], [20, 30], [60, 100]])
@pytest.mark.parametrize("q2,k2,alpha", [(-95, 95, None), (95, -95, None), (55, 55, 1e-33), (-50, -50, 1e30)])
def test_tiny_and_huge_factors_of_ordinary_scores(q2, k2, alpha, new, store, dtype, d):
    b = Batch(new, [50, 200], d=d, store=store, dtype=dtype)
    b.q = (b.q.float() * 2.0 ** q2).to(b.dt)
    b.k_all = (b.k_all.float() * 2.0 ** k2).to(b.dt)
    b.fill().check("softmax", alpha)
    b.check("silu", alpha)


@pytest.mark.parametrize("store,dtype,d,new,H", [("bf16", "bf16", 128, [1, 1], 2), ("bf16", "bf16", 64, [9, 12], 2), ("e4m3", "bf16", 128, [20, 30], 2),
                                                 ("bf16", "bf16", 128, [60, 100], 2), ("e4m3", "bf16", 64, [90, 40], 4),
                                                 ("f32", "f32", 64, [1, 1], 2), ("f32", "f32", 64, [9, 12], 2)])
@pytest.mark.parametrize("turn", ["tokens", "heads", "both"])
def test_strides_of_either_sign(turn, store, dtype, d, new, H):
    """Rows and heads that lie in memory from the last to the first (C callers)."""
    b = Batch(new, [50, 200], H=H, Hkv=2, d=d, store=store, dtype=dtype).fill()
    want, lse = b.run()
    axes = {"tokens": (0,), "heads": (1,), "both": (0, 1)}[turn]

    def rows(x):
        """The memory (to be kept) and the rows of x, turned."""
        m = x.flip(axes).contiguous()
        at, (t, h, _) = 0, m.stride()
        if 0 in axes:
            at, t = at + (x.shape[0] - 1) * t, -t
        if 1 in axes:
            at, h = at + (x.shape[1] - 1) * h, -h
        return m, raw._cache_rows(m.data_ptr() + at * m.element_size(), t, h)
    L, ref_, st = raw.lib(), b.cache._ref, torch.cuda.current_stream().cuda_stream
    kind, T, B = raw._DTYPE_ID[b.dt], sum(new), len(new)
    where = raw._cache_where(b.table.data_ptr(), b.off.data_ptr(), b.starts.data_ptr(), b.table.stride(0), b.table.shape[1], B)
    # written and read back
    k, v = (x[:T].cuda() for x in (b.k_all, b.v_all))
    mk, rk = rows(k)
    mv, rv = rows(v)
    before = gd.gdpa_cache_read(b.cache, T, b.table, b.off, b.starts, dtype=b.dt)
    assert L.gdpa_cache_write(ref_, kind, T, rk, rv, where, st) == 0
    straight = gd.gdpa_cache_read(b.cache, T, b.table, b.off, b.starts, dtype=b.dt)
    gd.gdpa_cache_write(b.cache, k, v, b.table, b.off, b.starts)
    for x, y in zip(straight, gd.gdpa_cache_read(b.cache, T, b.table, b.off, b.starts, dtype=b.dt)):
        assert torch.equal(x, y)
    mk, rk = rows(torch.zeros_like(k))
    mv, rv = rows(torch.zeros_like(v))
    assert L.gdpa_cache_read(ref_, kind, T, rk, rv, where, st) == 0
    assert torch.equal(mk.flip(axes), straight[0]) and torch.equal(mv.flip(axes), straight[1])
    gd.gdpa_cache_write(b.cache, *before, b.table, b.off, b.starts)
    # queries
    mq, rq = rows(b.q)
    o, l2 = torch.empty_like(b.q), torch.empty_like(lse)
    n = ctypes.c_int64()
    assert L.gdpa_cache_workspace(ref_, kind, T, H, B, ctypes.byref(n)) == 0
    work = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    attn = raw._cache_attn(0, 0, 0, raw.ACT["softmax"], d ** -0.5, 0)
    assert L.gdpa_cache_fwd(ref_, kind, T, H, rq, o.data_ptr(), l2.data_ptr(), where, attn, work.data_ptr(), n.value, st) == 0
    b.cache.check()
    assert torch.equal(o, want) and torch.equal(l2, lse)


def test_rows_behind_the_last_sample_stay():
    b = Batch([5, 3], [50, 20]).fill()
    q = torch.cat([b.q, b.q])
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    gd.gdpa_cache_softmax_fwd(b.cache, q, b.table, b.off, b.starts, o=o, lse=lse)
    w, wl = b.run()
    assert torch.equal(o[:8], w) and torch.equal(lse[:8], wl) and (o[8:] == 7).all() and (lse[8:] == 7).all()


def test_same_bits_every_time():
    b = Batch([1, 2, 7], [20000, 33, 500], H=8, Hkv=2, store="e4m3", page=64).fill()
    first = b.run()
    for _ in range(5):
        again = b.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("store,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("f32", "f32")])
def test_pages_outside_the_cache_are_not_read(store, dtype):
    b = Batch([1, 2], [100, 60], d=64, store=store, dtype=dtype).fill()
    good, _ = b.run()
    b.table_host[1, 1] = 1 << 20     # events 16 .. 31 of sample 1
    b.table = dev(b.table_host)
    o, _ = b.run()
    with pytest.raises(gd.GdpaError):
        b.cache.check()
    assert torch.equal(o[:1], good[:1])
    # as if these events were hidden
    keep = np.array([j for j in range(62) if not 16 <= j < 32])
    x = [orc.held(ref.to_f64(t), store) for t in (b.k_all, b.v_all)]
    k, v = ([t[101:][keep]] for t in x)
    for i in range(2):
        see = keep <= 60 + i
        want, _, size = orc.attend([0, 1], [see.sum() - 1], ref.to_f64(b.q[1 + i:2 + i]), [k[0][see]], [v[0][see]],
                                   64 ** -0.5, "softmax")
        check_o(o[1 + i:2 + i], want, size, "softmax", b)


def test_events_and_starts_outside_the_table():
    b = Batch([2, 1], [30, 60]).fill()
    good, _ = b.run()
    st = dev([-5, 60])
    o, lse = gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table, b.off, st)
    with pytest.raises(gd.GdpaError):
        b.cache.check()
    assert (o[:2] == 0).all() and torch.isinf(lse[:2]).all() and torch.equal(o[2:], good[2:])
    # starts that leave 32 bits behind
    o, lse = gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table, b.off, dev([2 ** 31 - 2, 60]), window=5)
    with pytest.raises(gd.GdpaError):
        b.cache.check()
    assert torch.equal(o[2:], gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table, b.off, b.starts, window=5)[0][2:])
    # a table too short for the events
    gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table[:, :3], b.off, b.starts)
    with pytest.raises(gd.GdpaError):
        b.cache.check()
    b.run()
    b.cache.check()


def test_a_run_of_them_as_a_server_makes_it():
    """Rotary positions, new rows written, scored, drafted continuations scored
    as a tree, all from one captured graph over growing histories."""
    H, Hkv, d, B, P = 4, 2, 64, 3, 16
    rope = gd.Rope(d)
    cache = gd.KVCache(40, Hkv, d, page=P, store="e4m3")
    table = dev(np.random.Generator(np.random.PCG64(1)).permutation(39).reshape(3, 13))
    off = dev(np.arange(B + 1))
    starts = dev([0, 5, 31])
    g = torch.Generator(device="cuda").manual_seed(3)
    hist_k = torch.randn((36, Hkv, d), generator=g, device="cuda").bfloat16()
    hist_v = torch.randn((36, Hkv, d), generator=g, device="cuda").bfloat16()
    hoff = dev([0, 0, 5, 36])
    gd.gdpa_cache_write(cache, gd.gdpa_rope_fwd(rope, hist_k, offsets=hoff), hist_v, table, hoff)
    x = [torch.zeros((B, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv)]

    def step():
        q, k = gd.gdpa_rope_fwd(rope, x[0], x[1], offsets=off, starts=starts)
        gd.gdpa_cache_write(cache, k, x[2], table, off, starts)
        return gd.gdpa_cache_softmax_fwd(cache, q, table, off, starts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    ks, vs = [hist_k[:0], hist_k[:5], hist_k[5:]], [hist_v[:0], hist_v[:5], hist_v[5:]]
    for _ in range(20):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ks = [torch.cat([a, x[1][i:i + 1]]) for i, a in enumerate(ks)]
        vs = [torch.cat([a, x[2][i:i + 1]]) for i, a in enumerate(vs)]
        n = [len(a) for a in ks]
        turned = gd.gdpa_rope_fwd(rope, torch.cat(ks), offsets=dev(offsets(n)))
        q = gd.gdpa_rope_fwd(rope, x[0], offsets=off, starts=starts)
        k64 = np.split(orc.held(ref.to_f64(turned), "e4m3"), np.cumsum(n)[:-1])
        v64 = np.split(orc.held(ref.to_f64(torch.cat(vs)), "e4m3"), np.cumsum(n)[:-1])
        want, wlse, size = orc.attend(np.arange(B + 1), [m - 1 for m in n], ref.to_f64(q), k64, v64, d ** -0.5, "softmax")

        class Of:
            dt, store, few = torch.bfloat16, "e4m3", True
        Of.d = d
        check_o(o, want, size, "softmax", Of)
        check_lse(lse, wlse)
        starts += 1
    cache.check()


def test_streams():
    """Calls on several streams at once, each with its own rows, one cache."""
    b = Batch([1, 4], [3000, 200], H=8, Hkv=2, store="e4m3", page=64).fill()
    want, lse = b.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = []
    for _ in range(6):
        for s in streams:
            out.append(gd.gdpa_cache_softmax_fwd(b.cache, b.q, b.table, b.off, b.starts, stream=s))
    torch.cuda.synchronize()
    for o, l2 in out:
        assert torch.equal(o, want) and torch.equal(l2, lse)


def test_refusals():
    b = Batch([2], [5], H=4, Hkv=2, d=64).fill()
    a = (b.cache, b.q, b.table, b.off, b.starts)
    f = gd.gdpa_cache_softmax_fwd
    with pytest.raises(ValueError):
        gd.gdpa_cache_fwd(*a, act="softmax")
    with pytest.raises(KeyError):
        f(*a, mask="none")
    with pytest.raises(ValueError):
        f(*a, mask="tree")
    with pytest.raises(ValueError):
        f(*a, parents=dev([0, 0]))
    with pytest.raises(ValueError):
        f(*a, mask="tree", parents=dev([0, 0, 0]))
    for kw in (dict(sinks=2), dict(window=-1), dict(window=3, sinks=-1), dict(alpha=float("nan")), dict(alpha=float("inf"))):
        with pytest.raises(gd.GdpaError) as e:
            f(*a, **kw)
        assert e.value.status == 1
    with pytest.raises(gd.GdpaError):
        f(b.cache, b.q[:, :3], *a[2:])           # 3 heads on 2 key heads
    for bad in (b.q.float(), b.q.half()):
        with pytest.raises(TypeError):
            f(b.cache, bad, *a[2:])
    for bad in (b.q[:, :, :32], b.q[0], b.q.cpu()):
        with pytest.raises(ValueError):
            f(b.cache, bad, *a[2:])
    with pytest.raises(ValueError):
        f(*a, o=torch.empty_like(b.q).transpose(0, 1))
    with pytest.raises(ValueError):
        f(*a, lse=torch.empty(2, 4, dtype=torch.bfloat16, device="cuda"))
