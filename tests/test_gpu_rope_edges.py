"""Rotary positions on the GPU at the edges of what its calls allow.  Helpers
and bounds as test_gpu_rope.py."""

import pytest

torch = pytest.importorskip("torch")

import recommender_model_attention_gb300 as gd  # noqa: E402
from oracle import rope as orc  # noqa: E402
from test_gpu_rope import check, rows  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(_):
    gd.build()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 3), (5, 1)])
def test_strides_that_are_never_stepped(T, H, layout, dt):
    """A single row's token stride and a single head's head stride say nothing
    about where values are: odd ones are taken too."""
    f = orc.frequencies(24)
    rope = gd.Rope(24, layout=layout)
    pos = torch.arange(T, device="cuda") + 3
    w = rows(6, 4, 41, dt)   # odd strides of tokens (164 + 41 = 205) and heads (41)
    store = torch.zeros(6 * 205, dtype=w.dtype, device="cuda")
    token, head = (205 if T == 1 else 164), (41 if H == 1 else 40)
    x = store.as_strided((T, H, 40), (token, head, 1))
    x.copy_(w[:T, :H, :40])
    want = gd.gdpa_rope_fwd(rope, x.contiguous(), positions=pos)
    check(want, x, pos.tolist(), f, layout)
    y = gd.gdpa_rope_fwd(rope, x, positions=pos)
    assert torch.equal(y, want)
    out = torch.zeros_like(store).as_strided((T, H, 40), (token, head, 1))
    assert torch.equal(gd.gdpa_rope_fwd(rope, x, positions=pos, q_out=out), want)
    a, b = gd.gdpa_rope_fwd(rope, x.contiguous(), x, positions=pos)
    assert torch.equal(a, want) and torch.equal(b, want)
    gd.gdpa_rope_fwd(rope, x, positions=pos, q_out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B", [255, 256, 257, 600, 1022, 1023, 1024, 2047, 2048, 5000])
def test_positions_counted_from_many_offsets(B, dt):
    """More offsets than a block has threads, and more than it counts through:
    the same bits as the positions given, also where many samples are empty."""
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    lens = torch.randint(0, 5, (B,), generator=g, device="cuda")
    lens[torch.rand(B, generator=g, device="cuda") < 0.3] = 0
    lens[B // 2] = 700   # over several blocks
    off = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), lens.cumsum(0)]).int()
    starts = torch.randint(-1000, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
    n = int(off[-1])
    x = rows(n + 9, 2, 64, dt)
    sample = torch.repeat_interleave(torch.arange(B, device="cuda"), lens)
    pos = torch.arange(n, device="cuda") - off[sample].long() + starts[sample].long()
    rope = gd.Rope(64)
    want = gd.gdpa_rope_fwd(rope, x[:n], positions=pos)
    got = gd.gdpa_rope_fwd(rope, x, offsets=off, starts=starts, q_out=torch.full_like(x, 3.25))
    assert torch.equal(got[:n], want) and torch.all(got[n:] == 3.25)
    at = [0, n // 3, n - 1]
    check(want[at], x[at], [int(pos[i]) for i in at], orc.frequencies(64), "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rows_past_32_bit_offsets(layout):
    """Values whose element offsets pass 2^31 and byte offsets 2^32, in place."""
    H, d = 8, 128
    T = 2 ** 31 // (H * d) + 77
    x = torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda")
    at = [0, 1, T // 2, T - 78, T - 77, T - 1]
    mine = rows(len(at), H, d, "bf16")
    x[at] = mine
    pos = torch.arange(T, device="cuda")
    assert gd.gdpa_rope_fwd(gd.Rope(d, layout=layout), x, positions=pos, q_out=x) is x
    check(x[at], mine, at, orc.frequencies(d), layout)
    assert int(torch.count_nonzero(x)) == int(torch.count_nonzero(x[at]))
