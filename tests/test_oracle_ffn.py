"""The plain forms of the gated block and of group-scaled 4-bit integers, against closed forms,
differences and value by value searches."""
import numpy as np
import pytest

from oracle import ffn_oracle as P


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations(act):
    from math import erf, exp, sqrt
    for v in (-30.0, -3.0, -0.5, 0.0, 1e-3, 0.7, 2.0, 25.0):
        got = float(P.act_value(np.array(v), act)[0])
        want = v / (1 + exp(-v)) if act == "silu" else v * (1 + erf(v / sqrt(2))) / 2
        assert abs(got - want) <= (1e-12 if act == "silu" else 2e-3)
        h = 1e-5
        diff = float(P.act_value(np.array(v + h), act)[0] - P.act_value(np.array(v - h), act)[0]) / (2 * h)
        assert abs(float(P.act_slope(np.array(v), act)[0]) - diff) < 1e-8
    v = np.linspace(-40, 40, 20001)
    assert np.abs(P.act_slope(v, act)[0]).max() < P.STEEP
    assert np.isfinite(P.act_slope(v, act)[0]).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_is_the_gradient(act):
    """Of f = sum(dy (h w_down)), by differences in every input."""
    rng = np.random.default_rng(3)
    off, rows, k, n, h = [0, 2, 2, 5], 5, 4, 3, 6
    x, dy = rng.standard_normal((rows, k)), rng.standard_normal((rows, h))
    wg, wu = rng.standard_normal((2, 3, k, n))
    wd = rng.standard_normal((3, n, h))

    def f(x, wg, wu):
        (hid, _), _, _ = P.glu(x, wg, wu, off, act)
        return (P.sums(hid, wd, off)[0] * dy).sum()

    _, (g, _), (u, _) = P.glu(x, wg, wu, off, act)
    (dg, _), (du, _) = P.glu_grad(dy, wd.transpose(0, 2, 1), g, u, off, act)
    dx, _ = P.glu_xgrad(dg, du, wg.transpose(0, 2, 1), wu.transpose(0, 2, 1), off)
    dwg = np.stack([x[a:b].T @ dg[a:b] for a, b in zip(off, off[1:])])
    dwu = np.stack([x[a:b].T @ du[a:b] for a, b in zip(off, off[1:])])
    for i, (v, d) in enumerate(((x, dx), (wg, dwg), (wu, dwu))):
        for at in np.ndindex(v.shape):
            lo, hi = [x, wg, wu], [x, wg, wu]
            lo[i], hi[i] = v.copy(), v.copy()
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            assert abs((f(*hi) - f(*lo)) / 2e-5 - d[at]) < 1e-7


def test_layout():
    q = np.random.default_rng(4).integers(0, 16, size=(3, 256)).astype(np.uint8)
    p = P.gq_pack(q)
    assert np.array_equal(P.gq_unpack(p), q)
    words = p.reshape(3, 2, 16, 4)
    # value 0 and 4 of a row lie in its first byte, value 8 in word 4, value 32 in word 1
    assert (words[:, 0, 0, 0] == (q[:, 0] | q[:, 4] << 4)).all()
    assert (words[:, 0, 4, 0] & 15 == q[:, 8]).all() and (words[:, 0, 1, 0] & 15 == q[:, 32]).all()
    assert (words[:, 1, 15, 3] >> 4 == q[:, 255]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_nearest_code(block, zeros, kind):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((20, 300)) * np.exp2(rng.integers(-8, 8, size=(20, 1)))).astype(np.float32)
    x[3] = np.abs(x[3])
    q, s, z = P.gq_quantize(x, block, kind, zeros)
    v, _ = P.gq_values(q, s, z if zeros else None, block)
    assert q.shape == (20, 384) and s.shape == z.shape == (20, 384 // block)
    wide = np.repeat(s.astype(np.float64), block, axis=1)[:, :300]
    zz = np.repeat(z.astype(np.float64), block, axis=1)[:, :300]
    lowest, highest = -zz * wide, (15 - zz) * wide
    best = np.clip(x.astype(np.float64), lowest, highest)       # the format's range of each block
    assert (np.abs(v[:, :300] - best) <= wide / 2 * (1 + 2.0 ** -20)).all()
    # the ends of a block lie within half a step of its range, one more for the rounded zero
    assert (np.abs(best - x) <= wide * 1.1).all()
    assert (v[:, 300:] == 0).all()
    if zeros:
        assert (z[3] == 0).all() and (v[3] >= 0).all()
    else:
        assert (z == 8).all()


def test_edges():
    x = np.zeros((6, 33), dtype=np.float32)
    x[1, 3], x[2, 3], x[3, 3], x[4, 32] = np.inf, np.nan, 2.0 ** -149, -7.0
    x[5, 0], x[5, 1] = 3e38, -3e38
    for zeros in (True, False):
        q, s, z = P.gq_quantize(x, 32, "bf16", zeros)
        v, _ = P.gq_values(q, s, z if zeros else None, 32)
        assert np.isnan(v[1:3, :32]).all() and not np.isnan(v[:, 32:]).any() and (v[3] == 0).all()
        assert np.isnan(v[5, 0]) == zeros                        # the range overflows, the magnitude does not
        assert abs(v[4, 32] + 7) <= 7 * 2.0 ** -8 and (v[0] == 0).all()
    q, s, z = P.gq_quantize(np.array([[1e7]], dtype=np.float32), 32, "fp16", True)
    assert np.isnan(s[0, 0]) and (q[0] == 0).all()


def test_scaled_sums():
    rng = np.random.default_rng(6)
    x, w = rng.standard_normal((5, 40)), rng.standard_normal((2, 7, 40)).astype(np.float32)
    qs = [P.gq_quantize(m, 32, "fp16", True) for m in w]
    vals = np.stack([P.gq_values(q, s, z, 32)[0] for q, s, z in qs])
    mags = np.stack([P.gq_values(q, s, z, 32)[1] for q, s, z in qs])
    y, err = P.gq_sums(x, vals, mags, [0, 3, 5], 32)
    for i in range(5):
        for n in range(7):
            g = 0 if i < 3 else 1
            want = sum(x[i, k] * vals[g, n, k] for k in range(40))
            assert abs(y[i, n] - want) < 1e-12 and err[i, n] > 0
            assert err[i, n] >= 2.0 ** -23 * abs(want)
