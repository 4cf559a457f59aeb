"""What a shared-prefix plan holds and refuses, without a GPU, beside
test_prefix_cpu.py: the lists that the kernels walk without checks of their own."""

import numpy as np
import pytest

import recommender_model_attention_gb300 as gd
from prefix_util import batch, orc
from test_prefix_cpu import _covered


def setup_module(_):
    gd.build()


@pytest.mark.parametrize("which", ["q_off", "kv_off", "prefix_off"])
@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 4095])
def test_rows_that_32_bit_steps_would_pass(which, rows):
    """A walk of 128-row blocks to the last row of 2^31 - 1 passes 2^31."""
    a = dict(q_off=[0, 2], kv_off=[0, 2], group_off=[0, 1], prefix_off=[0, 4])
    a[which] = [0, rows]
    with pytest.raises(gd.GdpaError) as e:
        gd.PrefixPlan(H=1, d=8, num_sms=4, host_only=True, **a)
    assert e.value.status == 2


BATCHES = {
    "ragged": batch([3, 1, 0, 40, 2, 130, 1], [2, 0, 5, 40, 6, 131, 0], [2, 0, 3, 2], [4, 7, 0, 300]),
    "single tokens": batch([1] * 70, [i % 9 for i in range(70)], [1, 69], [1000, 257]),
    "own keys only": batch([300, 1, 64, 60, 8], [290, 600, 64, 80, 512], [5], [0]),
    "many rows": batch([37] * 30 + [3], [5] * 30 + [700], [30, 1], [70, 0]),
    "many own rows": batch([1500, 7], [200, 2], [1, 1], [3, 0]),
    "keys without rows": batch([0, 0, 4], [40, 0, 3], [1, 1, 1], [5, 300, 0]),
    "one row": batch([1], [0], [1], [1]),
    "nothing": batch([], [], [], []),
}
SHAPES = pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 2), (40, 1), (4, 4)])
KINDS = pytest.mark.parametrize("d", [8, 64, 128])
WINDOWS = pytest.mark.parametrize("window,sms", [(0, 1), (0, 152), (37, 5), (1, 152), (2 ** 31 - 1, 20)])


def make(name, H, Hkv, d, window, sms):
    offs = BATCHES[name]
    plan = gd.PrefixPlan(*offs, H, d, kv_heads=Hkv, mask="causal_window" if window else "none",
                         window=window, num_sms=sms, host_only=True)
    return plan, offs


def small_samples(offs, r, d):
    """The planner's rule: few rows, few keys, few pairs of them."""
    lq, lk = np.diff(offs[0]) * r, np.diff(offs[1])
    ok = (lq > 0) & (lk > 0) & (lq <= 64) & (lk <= 512) & (lq * lk <= 4096)
    return np.nonzero(ok & (d in (64, 128)))[0]


@pytest.mark.parametrize("name", list(BATCHES))
@SHAPES
@KINDS
@WINDOWS
def test_forward_pieces_and_parts(name, H, Hkv, d, window, sms):
    """Every pair in one piece (small samples' in pieces of their own); the
    workspace's rows given out once; the CUDA cores' blocks and the 8-row units
    cover every row of what they walk once; the merge's records find the parts."""
    plan, offs = make(name, H, Hkv, d, window, sms)
    r = H // Hkv
    pieces, seg = _covered(plan, offs, H, Hkv, window)
    small = small_samples(offs, r, d)
    assert len(pieces) - seg[-1] == len(small) * Hkv
    part_rows, _, small8, warp_rows = plan.export_list("counts")[0].tolist()
    given = np.zeros(part_rows, dtype=np.int32)
    starts = {}
    for tok, na, nb, hk, k0, nk, flags, i0, j0, pa, pb, _ in pieces.tolist():
        for part, t0, n in ((pa, tok, na), (pb, tok if flags & 2 else tok + na, na if flags & 2 else nb)):
            if part >= 0:
                given[part:part + n * r] += 1
                assert part + n * r <= part_rows
                starts[part] = (t0, n, hk, flags & 1)
    assert np.all(given == 1)
    # the merge: a tile's prefix parts, and each token's own
    seen = np.zeros(part_rows, dtype=np.int32)
    own = plan.export_list("own")
    assert own.shape == (plan.Tq, 4)
    cover = np.zeros((plan.Tq, Hkv), dtype=np.int32)
    for tok, n, hk, part, layers, *_ in plan.export_list("tiles").tolist():
        cover[tok:tok + n, hk] += 1
        for i in range(layers):
            assert starts[part + i * n * r] == (tok, n, hk, 0)
            seen[part + i * n * r:part + (i + 1) * n * r] += 1
        for t in range(tok, tok + n):
            first, row0, lay, rows = own[t].tolist()
            for i in range(lay):
                at = first + (hk * lay + i) * rows
                t0, m, h, mine = starts[at]
                assert mine and h == hk and rows == m * r and t == t0 + row0 // r and row0 % r == 0
                seen[at + row0:at + row0 + r] += 1
    assert np.all(cover == 1) and np.all(seen == 1)
    # row blocks: 4 x rows a warp of a piece's slot
    done = [[np.zeros(na * r), np.zeros((na if fl & 2 else nb) * r)] for _, na, nb, _, _, _, fl, *_ in pieces.tolist()]
    for piece, sub in plan.export_list("blocks").tolist():
        first = (sub >> 1) * 4 * warp_rows
        rows = done[piece][sub & 1]
        assert first < len(rows) and pieces[piece, 9 + (sub & 1)] >= 0
        rows[first:first + 4 * warp_rows] += 1
    for (a, b), p in zip(done, pieces.tolist()):
        assert np.all(a == 1) and (np.all(b == 1) if p[10] >= 0 else not b.any())
    # small samples, whole and in 8 rows
    smalls = plan.export_list("smalls")
    q_off, kv_off = offs[0], offs[1]
    want = sorted((kv_off[b], kv_off[b + 1] - kv_off[b], q_off[b], q_off[b + 1] - q_off[b], hk, 1, 0, 0)
                  for b in small for hk in range(Hkv))
    assert sorted(map(tuple, smalls.tolist())) == want
    assert np.all(smalls[:small8, 3] * r <= 8) and np.all(smalls[small8:, 3] * r > 8)
    rows = {}
    for u in plan.export_list("eights").tolist():
        assert u[7] % 8 == 0 and u[7] < u[3] * r
        rows.setdefault(tuple(u[:7]) + (0,), []).append(u[7])
    assert sorted(rows) == want
    assert all(sorted(v) == list(range(0, u[3] * r, 8)) for u, v in rows.items())
    for b in small:   # the warp-level kernels: one tile, one part a head, from the first token on
        first, row0, lay, n = own[q_off[b]].tolist()
        assert row0 == 0 and lay == 1 and n == (q_off[b + 1] - q_off[b]) * r


@pytest.mark.parametrize("name", list(BATCHES))
@SHAPES
@KINDS
@WINDOWS
def test_backward_units(name, H, Hkv, d, window, sms):
    """Every (row, key) that is seen is in one unit, or one part of a unit; every
    key's gradient is written once; part numbers are used once, below their
    count, and joined in order; the same for the tensor cores' units with the
    small samples beside them."""
    plan, offs = make(name, H, Hkv, d, window, sms)
    r = H // Hkv
    units, joins = plan.export_list("units"), plan.export_list("joins")
    useg = plan.export_list("unit_seg")[:, 0]
    _, parts, _, _ = plan.export_list("counts")[0].tolist()
    assert len(useg) == sms + 1 and useg[0] == 0 and np.all(np.diff(useg) >= 0) and useg[-1] <= len(units)
    groups = list(orc.groups(*offs, "causal_window" if window else "none", window))
    q_off, kv_off, p_off = offs[0], offs[1], offs[3]
    by_part = {}
    for which in ("all units", "queues and small samples"):
        walked = units if which == "all units" else units[:useg[-1]]
        pre = np.zeros((Hkv, plan.Tq, plan.Tp), dtype=np.int8)
        own = np.zeros((Hkv, plan.Tq, max(1, plan.Tkv)), dtype=np.int8)
        wrote = [np.zeros((Hkv, plan.Tp), dtype=np.int32), np.zeros((Hkv, plan.Tkv), dtype=np.int32)]
        used = np.zeros(parts, dtype=np.int32)
        for k0, nk, tok, ntok, hk, flags, i0, j0 in walked.tolist():
            assert 0 < nk <= 128 and ntok >= 0 and tok + ntok <= plan.Tq
            mine, part = flags & 1, flags >> 8
            assert k0 + nk <= (plan.Tkv if mine else plan.Tp)
            (own if mine else pre)[hk, tok:tok + ntok, k0:k0 + nk] += 1
            if mine:
                b = int(np.searchsorted(kv_off, k0, side="right")) - 1
                assert k0 == kv_off[b] + j0 and k0 + nk <= kv_off[b + 1]
                assert tok == q_off[b] + i0 and tok + ntok <= q_off[b + 1]
            if part:
                assert part <= parts
                used[part - 1] += 1
                by_part[part - 1] = (k0, nk, hk, flags & 1, j0, tok, ntok)
            else:
                wrote[mine][hk, k0:k0 + nk] += 1
        assert np.all(used == 1)
        joined = []
        for k0, nk, first, n, hk, flags, i0, j0 in joins.tolist():
            wrote[flags & 1][hk, k0:k0 + nk] += 1
            joined += range(first, first + n)
            assert n > 1 and flags >> 8 == 0
            at = by_part[first][5]
            for i in range(first, first + n):   # ranges of the tokens, one behind the other
                assert by_part[i][:5] == (k0, nk, hk, flags & 1, j0) and by_part[i][5] == at and by_part[i][6] > 0
                at += by_part[i][6]
        assert sorted(joined) == list(range(parts))
        if which != "all units":
            for k0, nk, tok, ntok, hk, *_ in plan.export_list("smalls").tolist():
                own[hk, tok:tok + ntok, k0:k0 + nk] += 1
                wrote[1][hk, k0:k0 + nk] += 1
        assert np.all(wrote[0] == 1) and np.all(wrote[1] == 1)
        for rows, p, o, see in groups:
            for hk in range(Hkv):
                assert np.all(pre[hk][np.ix_(rows, p)] == 1)
                cover = own[hk][np.ix_(rows, o)]
                assert np.all(cover <= 1) and np.all(cover >= see[:, len(p):])
        assert pre.sum() == sum(len(rows) * len(p) for rows, p, _, _ in groups) * Hkv
    if name == "many rows" and sms > 1 and not window:
        assert parts > 1   # (a batch that is cut)


def test_lists_are_refused_where_they_do_not_fit():
    plan, _ = make("ragged", 1, 1, 64, 0, 4)
    import ctypes
    L, n, room = gd.lib(), ctypes.c_int64(), (ctypes.c_int32 * 4)()
    assert L.gdpa_prefix_export_list(plan.handle, 0, room, 0, ctypes.byref(n)) == 1 and n.value > 0
    assert L.gdpa_prefix_export_list(plan.handle, 0, None, 1 << 20, None) == 1
    assert L.gdpa_prefix_export_list(plan.handle, 8, room, 1, None) == 0
    for which in (-1, 9):
        assert L.gdpa_prefix_export_list(plan.handle, which, room, 1 << 20, None) == 1
    assert L.gdpa_prefix_export_list(None, 0, room, 1, None) == 1
    with pytest.raises(KeyError):
        plan.export_list("nothing")
