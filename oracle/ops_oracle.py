"""Plain 64-bit forms of the expert products and of microscaled 4-bit floating
point, from their definitions: numpy, no code shared with the HIP path.

4-bit format: 32 values share the scale 2^e, e = max(floor(log2 m) - 2, -127), m
the largest magnitude; a value is the nearest of +-{0 .5 1 1.5 2 3 4 6} * 2^e, of
two equally near ones the one with the even code, beyond 6 * 2^e the 6.  A block
with an infinity or a NaN has the scale byte 255 and zero codes.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK, PAD = 32, 128


def padded(cols: int) -> int:
    return -(-cols // PAD) * PAD


def mx_quantize(x: np.ndarray):
    """(codes [rows, kp] one per value, scale bytes [rows, kp / 32]) of x [rows, cols]."""
    rows, cols = x.shape
    kp = padded(cols)
    v = np.zeros((rows, kp))
    v[:, :cols] = x
    codes = np.zeros((rows, kp), dtype=np.uint8)
    scales = np.zeros((rows, kp // BLOCK), dtype=np.uint8)
    mid = (GRID[1:] + GRID[:-1]) / 2
    for b in range(kp // BLOCK):
        block = v[:, b * BLOCK:(b + 1) * BLOCK]
        finite = np.isfinite(block).all(axis=1)
        m = np.abs(np.where(finite[:, None], block, 0.0)).max(axis=1)
        e = np.where(m > 0, np.frexp(m)[1] - 1 - 2, -127)  # m = f * 2^ex with f in [.5, 1)
        e = np.maximum(e, -127)
        mag = np.abs(np.where(finite[:, None], block, 0.0)) * np.exp2(-e.astype(np.float64))[:, None]
        code = np.zeros(mag.shape, dtype=np.uint8)
        for i in range(7):  # past the middle between i and i + 1, or on it when i + 1 is even
            code += ((mag > mid[i]) | ((mag == mid[i]) & (i % 2 == 1))).astype(np.uint8)
        code |= np.where(np.signbit(block), 8, 0).astype(np.uint8)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.where(finite[:, None], code, 0)
        scales[:, b] = np.where(finite, e + 127, 255)
    codes[:, cols:] = 0
    return codes, scales


def mx_pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def mx_unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack((packed & 15, packed >> 4), axis=-1).reshape(*packed.shape[:-1], -1)


def mx_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Values of codes (one per value) and scale bytes."""
    v = np.where(codes >= 8, -GRID[codes & 7], GRID[codes & 7])
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def group_mm(x: np.ndarray, w: np.ndarray, offsets, out: np.ndarray):
    """out (changed in place) and the sums of the products' magnitudes: x [M, K], w [G, K, N]."""
    mag = np.zeros(out.shape)
    for g in range(w.shape[0]):
        a, b = offsets[g], offsets[g + 1]
        out[a:b] = x[a:b] @ w[g]
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[g])
    return out, mag


def group_wgrad(x: np.ndarray, dy: np.ndarray, offsets):
    g = len(offsets) - 1
    out = np.zeros((g, x.shape[1], dy.shape[1]))
    mag = np.zeros_like(out)
    for i in range(g):
        a, b = offsets[i], offsets[i + 1]
        out[i] = x[a:b].T @ dy[a:b]
        mag[i] = np.abs(x[a:b]).T @ np.abs(dy[a:b])
    return out, mag


def tolerance(want: np.ndarray, mag: np.ndarray, steps: int, unit: float) -> np.ndarray:
    """How far a product may be off: `steps` additions in 32 bits, each off by at most
    2^-23 of the magnitudes added up, then one rounding to the output's type (`unit`:
    half a step, relative), or half its smallest step (2^-25 in fp16)."""
    sums = (steps + 8) * 2.0 ** -23 * mag
    return sums + unit * (np.abs(want) + sums) + 2.0 ** -25 * (unit == 2.0 ** -11) + 2.0 ** -120
