"""Plain forms of the gated feed-forward block, of its backward pass and of 4-bit integer
weights with group scales, from their definitions: numpy, no code shared with the HIP path.

Values in 64 bits with the error that a computation in 32 bits may have: sums of n terms are
off by at most n 2^-23 of the magnitudes added up; the logistic function of z, whose argument
has been rounded a few times, is off by (|z| + 1) 2^-20 relative, since exp turns an absolute
error of its argument into a relative one; neither activation is steeper than 1.13.
"""
from __future__ import annotations

import numpy as np

PAD = 128
SILU, GELU = "silu", "gelu"
STEEP = 1.13


def _z(v, act):
    """Argument of the logistic function and its derivative."""
    if act == SILU:
        return v, np.ones_like(v)
    c = 2 * np.sqrt(2 / np.pi)
    return c * (v + 0.044715 * v ** 3), c * (1 + 3 * 0.044715 * v ** 2)


def _logistic(z):
    e = np.exp(-np.abs(z))
    return np.where(z < 0, e, 1.0) / (1 + e)


def act_value(v, act):
    """(act(v), error of its evaluation in 32 bits)."""
    z, _ = _z(v, act)
    with np.errstate(invalid="ignore"):
        a = np.where(v == -np.inf, 0.0, v * _logistic(z))        # its limit
    return a, np.abs(a) * (np.minimum(np.abs(z), 100) + 1) * 2.0 ** -20


def act_slope(v, act):
    """(act'(v), error of its evaluation in 32 bits)."""
    z, dz = _z(v, act)
    s, t = _logistic(z), v * _logistic(z) * _logistic(-z) * dz
    return s + t, (s + np.abs(t)) * (np.minimum(np.abs(z), 100) + 2) * 2.0 ** -19


def rounding(want, err, unit):
    """Error after one rounding to the output's type (`unit`: half a step, relative; fp16 has
    a smallest step)."""
    return err + unit * (np.abs(want) + err) + 2.0 ** -25 * (unit == 2.0 ** -11) + 2.0 ** -110


def sums(x, w, offsets, steps=None):
    """x [M, K] times w[g] [K, N] on the rows of every group, and the error of sums in 32 bits."""
    out, err = np.zeros((x.shape[0], w[0].shape[1])), np.zeros((x.shape[0], w[0].shape[1]))
    n = x.shape[1] if steps is None else steps
    for g in range(len(offsets) - 1):
        a, b = offsets[g], offsets[g + 1]
        out[a:b] = x[a:b] @ w[g]
        err[a:b] = (n + 8) * 2.0 ** -23 * (np.abs(x[a:b]) @ np.abs(w[g]))
    return out, err


def gated(g, eg, u, eu, act):
    """act(g) u and its error in 32 bits."""
    a, ea = act_value(g, act)
    ea = ea + STEEP * eg
    h = a * u
    return h, ea * (np.abs(u) + eu) + np.abs(a) * eu + np.abs(h) * 2.0 ** -22


def glu(x, wg, wu, offsets, act):
    """(h, G, U), each with its error in 32 bits."""
    g, eg = sums(x, wg, offsets)
    u, eu = sums(x, wu, offsets)
    return gated(g, eg, u, eu, act), (g, eg), (u, eu)


def glu_grad(dy, wd, gate, up, offsets, act):
    """(dG, dU), each with its error in 32 bits."""
    d, ed = sums(dy, wd, offsets)
    a, ea = act_value(gate, act)
    s, es = act_slope(gate, act)
    dg, du = d * up * s, d * a
    return ((dg, np.abs(up) * (ed * (np.abs(s) + es) + np.abs(d) * es) + np.abs(dg) * 2.0 ** -21),
            (du, ed * (np.abs(a) + ea) + np.abs(d) * ea + np.abs(du) * 2.0 ** -21))


def glu_xgrad(dg, du, wg, wu, offsets):
    k = dg.shape[1]
    a, ea = sums(dg, wg, offsets, 2 * k)
    b, eb = sums(du, wu, offsets, 2 * k)
    return a + b, ea + eb


# ------------------------------------------------- 4-bit integers with group scales

def padded(cols: int) -> int:
    return -(-cols // PAD) * PAD


def to_scale_type(s: np.ndarray, kind: str) -> np.ndarray:
    """fp32 values rounded to bf16 or fp16 (ties to even), below 2^-126 to zero."""
    s = s.astype(np.float32)
    if kind == "fp16":
        with np.errstate(over="ignore"):
            return s.astype(np.float16).astype(np.float32)
    bits = s.view(np.uint32).astype(np.uint64)
    r = ((bits + 0x7fff + ((bits >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    r = np.where(np.isnan(s), s, r)
    return np.where(r < 2.0 ** -126, np.float32(0), r)


def gq_quantize(x: np.ndarray, block: int, kind: str, zeros: bool):
    """(codes [rows, kp] one per value, scales [rows, kp / block] fp32 (NaN: a block that is not
    finite), zeros of the same shape) of x [rows, cols] in fp32; quotients in fp32."""
    rows, cols = x.shape
    kp = padded(cols)
    v = np.zeros((rows, kp), dtype=np.float32)
    v[:, :cols] = x
    v = v.reshape(rows, kp // block, block)
    finite = np.isfinite(v).all(axis=2)
    c = np.where(finite[:, :, None], v, np.float32(0))
    lo, hi = np.minimum(c.min(axis=2), 0), np.maximum(c.max(axis=2), 0)
    with np.errstate(over="ignore"):
        s = ((hi - lo) * (np.float32(1) / np.float32(15)) if zeros
             else np.abs(c).max(axis=2) * (np.float32(1) / np.float32(7)))
    s = to_scale_type(s, kind)
    bad = ~finite | ~np.isfinite(s)
    d = np.where(bad | (s == 0), np.float32(1), s)

    def over(n, d):
        return np.where(s.reshape(d.shape) > 0, n / d, np.float32(0)).astype(np.float32)

    z = np.clip(np.rint(over(-lo, d)), 0, 15) if zeros else np.full(s.shape, np.float32(8))
    q = np.clip(np.rint(np.where(s[:, :, None] > 0, c / d[:, :, None], 0)) + z[:, :, None], 0, 15)
    z = np.where(bad, 0, z).astype(np.uint8)
    q = np.where(bad[:, :, None], 0, q).astype(np.uint8)
    return q.reshape(rows, kp), np.where(bad, np.float32("nan"), s), z


def gq_pack(q: np.ndarray) -> np.ndarray:
    """Bytes of codes [.., kp], by the layout's definition, value by value."""
    kp = q.shape[-1]
    out = np.zeros(q.shape[:-1] + (kp // 2,), dtype=np.uint8)
    for base in range(0, kp, 128):
        for w in range(16):
            qq, u = w // 4, w % 4
            for b in range(4):
                v = base + 32 * u + 8 * qq + b
                out[..., base // 2 + 4 * w + b] = q[..., v] | (q[..., v + 4] << 4)
    return out


def gq_unpack(packed: np.ndarray) -> np.ndarray:
    kp = packed.shape[-1] * 2
    out = np.zeros(packed.shape[:-1] + (kp,), dtype=np.uint8)
    for base in range(0, kp, 128):
        for w in range(16):
            qq, u = w // 4, w % 4
            for b in range(4):
                v, byte = base + 32 * u + 8 * qq + b, packed[..., base // 2 + 4 * w + b]
                out[..., v], out[..., v + 4] = byte & 15, byte >> 4
    return out


def gq_values(q: np.ndarray, scales: np.ndarray, zeros, block: int):
    """Values [.., kp] in 64 bits, and s (q + z), the magnitudes that a product adds up."""
    s = np.repeat(scales.astype(np.float64), block, axis=-1)
    z = np.repeat(zeros.astype(np.float64), block, axis=-1) if zeros is not None else 8.0
    return s * (q - z), np.abs(s) * (q + z)


def gq_sums(x, w, mag, offsets, block):
    """x [M, K] times w[g]^T ([G, N, kp] values and magnitudes), and the error of the sums in 32
    bits: the terms of x q and of x, and three roundings a block."""
    rows, k = x.shape
    out, err = np.zeros((rows, w.shape[1])), np.zeros((rows, w.shape[1]))
    steps = k + 3 * (k // block + 1) + 8
    for g in range(len(offsets) - 1):
        a, b = offsets[g], offsets[g + 1]
        out[a:b] = x[a:b] @ w[g, :, :k].T
        err[a:b] = steps * 2.0 ** -23 * (np.abs(x[a:b]) @ mag[g, :, :k].T)
    return out, err
