"""Rotary positions on the GPU against exact angles and float64 products.

Error bounds, per value with s = A (|a| + |b|) of its pair (A the amplitude):

* float32 rows: the angle is off by at most 2^-33 turns and one rounding to
  float32 of at most half a turn (together under 1.0e-7 rad), sine and cosine
  by an ulp (2^-23), their product with A, the two products and the sum by
  2^-24 each, in total under 1.0e-7 + 1.2e-7 + 3 * 6.0e-8 = 4.0e-7 < 2^-21 s.
* bf16 rows: the hardware sine and cosine are off by 2^-21.2 on [-pi, pi]
  (4.2e-7), their argument by 3e-7, the products as above: under 2^-20 s; then
  one rounding to bf16 (8 significant bits): half a step, 2^-8 of the value.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from oracle import ref  # noqa: E402
from oracle import rope as orc  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def setup_module(_):
    gd.build()


def check(got, x, pos, freqs, layout, scale=1.0, inverse=False):
    want, s = orc.apply(ref.to_f64(x), pos, freqs, layout, scale, inverse)
    err = np.abs(ref.to_f64(got) - want)
    if x.dtype == torch.float32:
        bound = 2.0 ** -21 * scale * s
    else:
        bound = 2.0 ** -20 * scale * s * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert np.all(err <= bound), "worst %.3g of its bound" % np.max(err / np.maximum(bound, 1e-300))


def rows(T, H, d, dt, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, H, d), generator=g, device="cuda").to(DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (40, 40), (40, 24), (32, 2),
                                   (20, 6), (96, 90), (128, 120), (6, 6)])
def test_sizes_layouts(dt, layout, d, rot):
    f = orc.frequencies(rot)
    q, k = rows(37, 3, d, dt), rows(37, 2, d, dt, 1)
    pos = torch.arange(37, device="cuda", dtype=torch.int32) * 13 - 100
    rope = gd.Rope(rot, layout=layout)
    yq, yk = gd.gdpa_rope_fwd(rope, q, k, positions=pos)
    check(yq, q, pos.tolist(), f, layout)
    check(yk, k, pos.tolist(), f, layout)
    # alone, in place, and back
    assert torch.equal(gd.gdpa_rope_fwd(rope, k, positions=pos), yk)
    z = q.clone()
    assert gd.gdpa_rope_fwd(rope, z, positions=pos, q_out=z) is z and torch.equal(z, yq)
    dq, dk = gd.gdpa_rope_bwd(rope, yq, yk, positions=pos)
    check(dq, yq, pos.tolist(), f, layout, inverse=True)
    check(dk, yk, pos.tolist(), f, layout, inverse=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
def test_far_positions(dt, bits):
    rng = np.random.default_rng(3)
    f = np.array([1.0, 0.75, 3e-3, -0.5, 1e-7, 2.0, 0.0, 1000.0])
    top = 2 ** 31 if bits == torch.int32 else 2 ** 34
    pos = rng.integers(-top, top, size=64)
    pos[:3] = [top - 1, -top, 0]
    x = rows(64, 2, 16, dt)
    rope = gd.Rope(16, freqs=f, scale=1.25)
    # 2^-65 turns per position of frequency rounding: 2^-31 turns at 2^34,
    # another 3e-9 rad, inside the slack of the bounds above
    check(gd.gdpa_rope_fwd(rope, x, positions=torch.from_numpy(pos).cuda().to(bits)), x,
          pos.tolist(), f, "half", 1.25)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "by_parts"])
def test_scaled(scaling):
    kw = dict(base=10000.0, scaling=scaling, factor=4.0, orig_len=2048.0, lo=1.0, hi=32.0)
    x = rows(50, 2, 64, "f32")
    pos = list(range(0, 5000, 100))
    rope = gd.Rope(64, scale=1.1386294361119891, **kw)
    y = gd.gdpa_rope_fwd(rope, x, positions=torch.tensor(pos, device="cuda"))
    # frequencies from two maths libraries: 4 ulp at position 5000, 4e-12 rad
    check(y, x, pos, orc.frequencies(64, **kw), "half", float(np.float32(1.1386294361119891)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[0], [1], [0, 3, 0, 0, 17, 1, 0], [300, 2, 45], [5] * 200])
def test_positions_from_offsets(dt, lens):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(off[-1]) + 6   # rows behind the last sample stay as they are
    f = orc.frequencies(32)
    rope = gd.Rope(32)
    x = rows(T, 3, 48, dt)
    starts = np.arange(len(lens), dtype=np.int32) * 1000 - 7
    for st in (None, starts):
        out = torch.full_like(x, 3.25)
        y = gd.gdpa_rope_fwd(rope, x, offsets=torch.from_numpy(off).cuda(), q_out=out,
                             starts=None if st is None else torch.from_numpy(st).cuda())
        b = np.repeat(np.arange(len(lens)), lens)
        pos = np.arange(T - 6) - off[:-1][b] + (0 if st is None else st[b])
        if T > 6:
            check(y[:T - 6], x[:T - 6], pos.tolist(), f, "half")
        assert torch.all(y[T - 6:] == 3.25)
    assert torch.all(gd.gdpa_rope_fwd(rope, x[:6], offsets=torch.zeros(1, dtype=torch.int32, device="cuda"),
                                      q_out=torch.full_like(x[:6], 2.0)) == 2.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides(dt, layout):
    """Parts of a packed projection, head-major rows and unaligned column views."""
    f = orc.frequencies(24)
    rope = gd.Rope(24, layout=layout)
    pos = torch.arange(29, device="cuda")
    w = rows(29, 7, 40, dt)
    q, k = w[:, :4], w[:, 4:6]
    yq, yk = gd.gdpa_rope_fwd(rope, q, k, positions=pos)
    check(yq, q, pos.tolist(), f, layout)
    check(yk, k, pos.tolist(), f, layout)
    keep = w.clone()
    gd.gdpa_rope_fwd(rope, q, k, positions=pos, q_out=q, k_out=k)   # in place, V untouched
    assert torch.equal(w[:, :4], yq) and torch.equal(w[:, 4:6], yk) and torch.equal(w[:, 6], keep[:, 6])
    hm = rows(5, 29, 40, dt).transpose(0, 1)
    check(gd.gdpa_rope_fwd(rope, hm, positions=pos), hm, pos.tolist(), f, layout)
    odd = rows(29, 3, 50, dt)[..., 2:42]
    check(gd.gdpa_rope_fwd(rope, odd, positions=pos), odd, pos.tolist(), f, layout)
    one = rows(29, 3, 51, dt)[..., 1:41]   # rows of odd alignment
    if layout == "half":
        check(gd.gdpa_rope_fwd(rope, one, positions=pos), one, pos.tolist(), f, layout)
    else:
        with pytest.raises(gd.GdpaError):
            gd.gdpa_rope_fwd(rope, one, positions=pos)
    wide = rows(1, 3, 40, dt).expand(29, 3, 40)   # one row at many positions
    check(gd.gdpa_rope_fwd(rope, wide, positions=pos), wide, pos.tolist(), f, layout)


def test_gradient_is_the_adjoint_and_the_difference_quotient():
    f = orc.frequencies(16)
    rope = gd.Rope(16, scale=1.5)
    x, dy = rows(11, 2, 20, "f32"), rows(11, 2, 20, "f32", 1)
    pos = torch.arange(11, device="cuda") * 5
    y = gd.gdpa_rope_fwd(rope, x, positions=pos)
    dx = gd.gdpa_rope_bwd(rope, dy, positions=pos)
    check(dx, dy, pos.tolist(), f, "half", 1.5, inverse=True)
    a, b = float((y.double() * dy.double()).sum()), float((x.double() * dx.double()).sum())
    # every term within the float32 bound of this file, summed
    size = float((x.double().abs().sum() * dy.double().abs().max()))
    assert abs(a - b) <= 2 * 2.0 ** -21 * 1.5 * 2 * size
    # the map is linear: its difference along any direction is its value there
    e = rows(11, 2, 20, "f32", 2)
    diff = (gd.gdpa_rope_fwd(rope, x + e, positions=pos).double() - y.double() * 1.0)
    want = gd.gdpa_rope_fwd(rope, (x + e) - x, positions=pos).double()
    top = float(x.abs().max() + e.abs().max())
    assert float((diff - want).abs().max()) <= 3 * 2.0 ** -21 * 1.5 * 2 * top


@pytest.mark.parametrize("T,H,Hk", [(1, 1, 0), (1, 16, 16), (3, 200, 1), (5000, 8, 8), (70001, 1, 1),
                                    (20000, 16, 16)])
def test_row_and_head_counts(T, H, Hk):
    """Every split of heads over threads, checked on sampled rows."""
    f = orc.frequencies(64)
    rope = gd.Rope(64)
    q = rows(T, H, 64, "bf16")
    k = rows(T, Hk, 64, "bf16", 1) if Hk else None
    pos = torch.arange(T, device="cuda")
    y = gd.gdpa_rope_fwd(rope, q, k, positions=pos)
    y = y if Hk else (y,)
    at = sorted({0, T // 3, T // 2, T - 1})
    for x, z in zip((q, k), y):
        check(z[at], x[at], at, f, "half")
    if Hk == H and T > 1000:   # the whole tensor: a turn and its inverse give back the rows
        back = gd.gdpa_rope_bwd(rope, y[0], y[1], positions=pos)
        for x, z in zip((q, k), back):
            # two roundings to bf16 (2^-8 each) of a pair no longer than r = sqrt(2) max|x|:
            # the first reaches a value through both its columns, sqrt(2) r, the second adds r
            assert float((x.float() - z.float()).abs().max()) <= 4 * 2.0 ** -8 * float(x.float().abs().max())


def test_no_rows_and_no_heads():
    rope = gd.Rope(8)
    none = torch.empty((0, 3, 16), device="cuda")
    p = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert gd.gdpa_rope_fwd(rope, none, positions=p).shape == none.shape
    q, k = rows(4, 2, 16, "f32"), torch.empty((4, 0, 16), device="cuda")
    a, b = gd.gdpa_rope_fwd(rope, q, k, positions=torch.arange(4, device="cuda"))
    assert torch.equal(a, gd.gdpa_rope_fwd(rope, q, positions=torch.arange(4, device="cuda")))
    assert b.shape == k.shape


def test_special_values_stay_in_their_pair():
    x = rows(4, 2, 16, "f32")
    x[1, 0, 3] = float("nan")
    x[2, 1, 9] = float("inf")
    y = gd.gdpa_rope_fwd(gd.Rope(16), x, positions=torch.arange(4, device="cuda"))
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[1, 0, [3, 11]] = True
    bad[2, 1, [1, 9]] = True
    assert not torch.isfinite(y[bad]).any() and torch.isfinite(y[~bad]).all()


def test_stream_and_graph():
    rope = gd.Rope(64)
    x, out = rows(300, 4, 64, "bf16"), torch.zeros((300, 4, 64), device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    want = gd.gdpa_rope_fwd(rope, x, offsets=off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gd.gdpa_rope_fwd(rope, x, offsets=off, q_out=out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gd.gdpa_rope_fwd(rope, x, offsets=off, q_out=out)
    x.copy_(rows(300, 4, 64, "bf16", 9))
    off.copy_(torch.tensor([0, 7, 250], dtype=torch.int32))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    want = gd.gdpa_rope_fwd(rope, x, offsets=off)
    assert torch.equal(out[:250], want[:250]) and torch.all(out[250:] == 0)


def test_refusals():
    rope = gd.Rope(8)
    q, p = rows(4, 2, 16, "f32"), torch.arange(4, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bad = [dict(), dict(positions=p, offsets=off), dict(positions=p.float()), dict(positions=p[:3]),
           dict(positions=p.cpu()), dict(positions=torch.arange(8, device="cuda")[::2]),
           dict(offsets=off.long()), dict(offsets=off, starts=off), dict(positions=p, starts=off),
           dict(offsets=off.cpu()), dict(positions=p, k_out=q), dict(positions=p, q_out=q[:3]),
           dict(positions=p, q_out=q[:1].expand(4, 2, 16))]
    for kw in bad:
        with pytest.raises(ValueError):
            gd.gdpa_rope_fwd(rope, q, **kw)
    for t in (q.half(), q.double()):
        with pytest.raises(TypeError):
            gd.gdpa_rope_fwd(rope, t, positions=p)
    with pytest.raises(TypeError):
        gd.gdpa_rope_fwd(rope, q, q.bfloat16(), positions=p)
    with pytest.raises(ValueError):
        gd.gdpa_rope_fwd(rope, q.cpu(), positions=p)
    with pytest.raises(ValueError):
        gd.gdpa_rope_fwd(rope, q[0], positions=p)
    with pytest.raises(ValueError):
        gd.gdpa_rope_fwd(rope, q.transpose(1, 2), positions=p)
    with pytest.raises(gd.GdpaError):   # more columns turn than there are
        gd.gdpa_rope_fwd(gd.Rope(32), q, positions=p)
