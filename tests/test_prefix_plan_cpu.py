"""What a shared-prefix plan holds and refuses, without a GPU, beside
test_prefix_cpu.py."""

import pytest

import recommender_model_attention_gb300 as gd


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
