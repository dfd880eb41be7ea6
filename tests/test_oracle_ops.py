"""The plain forms of the 4-bit format and of the grouped products, against
closed forms and value by value searches."""
import numpy as np
import pytest

from oracle import ops_oracle as P


def test_every_grid_value_survives():
    row = np.concatenate((P.GRID, -P.GRID, P.GRID, -P.GRID))[None]
    for e in (-125, -10, 0, 7, 120):
        c, s = P.mx_quantize(row * 2.0 ** e)
        assert s[0, 0] == e + 127 and (s[0, 1:] == 0).all()
        assert np.array_equal(P.mx_values(c, s)[:, :32], row * 2.0 ** e)


def test_nearest_with_ties_to_even():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-20, 20, size=(40, 1)))
    x[0, :8] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5]
    x[0, 8:32] = 0
    c, s = P.mx_quantize(x)
    assert c[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6]
    v = P.mx_values(c, s)[:, :64]
    for r in range(40):
        for k in range(64):
            sc = 2.0 ** (int(s[r, k // 32]) - 127)
            best = min(abs(abs(x[r, k]) - g * sc) for g in P.GRID)
            assert abs(abs(x[r, k]) - abs(v[r, k])) == best
        for b in (0, 1):
            m = np.abs(x[r, 32 * b:32 * b + 32]).max()
            assert 4 <= m / 2.0 ** (int(s[r, b]) - 127) < 8


def test_edges():
    x = np.zeros((6, 33))
    x[1, 3], x[2, 3], x[3, 3] = np.inf, np.nan, 2.0 ** -149
    x[4, 32] = 7.9
    x[5, 0], x[5, 1] = -0.0, 4.0
    c, s = P.mx_quantize(x)
    assert c.shape == (6, 128) and s.shape == (6, 4)
    assert s[:, 0].tolist() == [0, 255, 255, 0, 0, 127] and s[4, 1] == 127
    v = P.mx_values(c, s)
    assert np.isnan(v[1, :32]).all() and np.isnan(v[2, :32]).all() and not np.isnan(v[:, 32:]).any()
    assert v[4, 32] == 6.0 and c[5, 0] == 8 and v[3, 3] == 0
    assert np.array_equal(P.mx_unpack(P.mx_pack(c)), c)


@pytest.mark.parametrize("offsets", [[0, 3, 3, 7], [0, 0, 0, 5]])
def test_grouped_products(offsets):
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((8, 5)), rng.standard_normal((3, 5, 4))
    y, mag = P.group_mm(x, w, offsets, np.full((8, 4), 9.0))
    g, _ = P.group_wgrad(x, y, offsets)
    for i in range(8):
        e = next((j for j in range(3) if offsets[j] <= i < offsets[j + 1]), None)
        for n in range(4):
            want = 9.0 if e is None else sum(x[i, k] * w[e, k, n] for k in range(5))
            assert abs(y[i, n] - want) < 1e-12
    for e in range(3):
        want = sum((np.outer(x[i], y[i]) for i in range(offsets[e], offsets[e + 1])), np.zeros((5, 4)))
        assert np.allclose(g[e], want, atol=1e-12, rtol=0)
    assert (mag >= np.abs(np.where(mag > 0, y, 0)) - 1e-12).all()
