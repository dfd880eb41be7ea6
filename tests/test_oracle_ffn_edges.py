"""The plain forms of the gated block and of 4-bit integers at the ends of their ranges."""
import numpy as np
import pytest

from oracle import ffn_oracle as P


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_far_out(act):
    far = np.array([-np.inf, -1e30, np.inf, np.nan])
    with np.errstate(over="ignore", invalid="ignore"):
        a, _ = P.act_value(far, act)
    assert a[0] == 0 and a[1] == 0 and a[2] == np.inf and np.isnan(a[3])
