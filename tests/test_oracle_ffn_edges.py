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


@pytest.mark.parametrize("kind,bits", [("bf16", 8), ("fp16", 11)])
@pytest.mark.parametrize("zeros", [True, False])
def test_scales_are_as_near_as_their_type_has_them(zeros, kind, bits):
    """Against the quotient in 64 bits: half a step, and three roundings to 24 bits (of the range, of
    the reciprocal and of the product), 3 2^-24 of a value that is less than 2^bits steps."""
    rng = np.random.default_rng(12)
    x = (rng.standard_normal((20000, 32)) * 0.02).astype(np.float32)
    _, s, _ = P.gq_quantize(x, 32, kind, zeros)
    v = x.astype(np.float64)
    want = ((np.maximum(v.max(1), 0) - np.minimum(v.min(1), 0)) / 15 if zeros else np.abs(v).max(1) / 7)
    step = 2.0 ** (np.floor(np.log2(want)) + 1 - bits)
    assert (np.abs(s[:, 0].astype(np.float64) - want) <= (0.5 + 3 * 2.0 ** (bits - 24)) * step).all()
