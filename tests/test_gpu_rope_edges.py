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
