"""The gated block and the 4-bit integer operators at the ends of their types' range, against the
definitions in 64 bits of oracle/ffn_oracle.py."""
import numpy as np
import pytest
import torch

from oracle import ffn_oracle as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import lossless_weight_compression_amd as L  # noqa: E402
from lossless_weight_compression_amd.layer import GqMatrix  # noqa: E402
from tests.gpu_harness import say  # noqa: E402
from tests.test_gpu_ffn import (BF, F16, F32, TYPES, check_glu, check_gq, check_grad, check_xgrad, close, host,  # noqa: E402
                                np64, off_dev, rand)  # noqa: E402


# ------------------------------------------------------ 4-bit values of the largest scales

def rounded_once(vals, dtype):
    """Values in 64 bits, exact products of 5 and 11 bits at most, in a type of the result."""
    return torch.from_numpy(vals).to(F32).to(dtype)


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 3, 128), (2, 5, 256), (1, 4, 100), (3, 2, 33)])
def test_largest_values_come_back(shape, dtype, zeros):
    """Blocks whose scale is finite while 8 or 15 times the scale is not."""
    say(f"[gpu] largest values {shape} {dtype} zeros={zeros}")
    x = torch.zeros(shape, dtype=F32)
    # with zeros the range, without them the magnitude has to be a number
    top = (-3.38e38, -3.3e38, -2e38) if zeros else (3e38, -3.38e38, 2.99e38)
    for r in range(shape[1]):
        x[:, r, 0] = top[r % 3]
        x[:, r, 1] = 0.3 * top[r % 3] if zeros else -0.3 * top[r % 3]
    x = x.to(dtype).cuda()
    q = GqMatrix(*shape[1:], groups=shape[0], block=32, with_zeros=zeros).quantize(x)
    codes, s, z = host(q)
    assert np.isfinite(s).all()
    with np.errstate(over="ignore"):
        vals = P.gq_values(codes, s, z, 32)[0][..., :shape[2]]
    for out in (BF, F16, F32):
        back = torch.full(shape, 7.0, dtype=out, device="cuda")
        q.dequantize(back)
        assert torch.equal(back.cpu(), rounded_once(vals, out)), out
        assert (back[..., 2:] == 0).all()
    # half a step and the scale's own rounding
    assert (np.abs(np64(q.dequantize(torch.empty(shape, dtype=F32, device="cuda"))) - np64(x)) <= 0.51 * s.max()).all()


@pytest.mark.parametrize("cols", [128, 160])
def test_every_code_of_a_large_scale(cols):
    """All codes with all zeros, scales from the smallest to the largest of their type."""
    rows = 16
    codes = np.tile(np.arange(cols) % 16, (1, rows, 1)).astype(np.uint8)
    codes = np.concatenate([codes, np.zeros((1, rows, P.padded(cols) - cols), np.uint8)], axis=2)
    zeros = np.tile(np.arange(rows, dtype=np.uint8)[None, :, None], (1, 1, P.padded(cols) // 32))
    for dtype, some in ((BF, (2.0 ** -133, 2.0 ** -126, 1.5, 2.2e37, 2.4e37, 4e37, 3e38)),
                        (F16, (2.0 ** -24, 2.0 ** -14, 3.0, 4400.0, 65504.0))):
        for s in some:
            scales = torch.full((1, rows, P.padded(cols) // 32), s, dtype=dtype, device="cuda")
            q = GqMatrix(rows, cols, block=32, codes=torch.from_numpy(P.gq_pack(codes)).cuda(), scales=scales,
                         zeros=torch.from_numpy(zeros).cuda())
            vals = P.gq_values(codes, scales.double().cpu().numpy(), zeros, 32)[0][..., :cols]
            for out in (BF, F16, F32):
                back = torch.full((1, rows, cols), 7.0, dtype=out, device="cuda")
                q.dequantize(back)
                assert torch.equal(back.cpu(), rounded_once(vals, out)), (dtype, s, out)


# -------------------------------------------------------------- gates without a number

# rows, columns that make few rows to a group, mid and large tiles of one matrix
PLACES = [(1, 64), (90, 72), (300, 264), (700, 130), (4096, 2304)]
INF = float("inf")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,n", PLACES)
def test_gates_at_infinity(rows, n, act):
    """act(-inf) and act'(-inf) are 0, their limits; act(inf) is inf, act'(inf) 1; NaN stays."""
    say(f"[gpu] gates at infinity {rows} {n} {act}")
    k = 8
    for dtype, kept in ((BF, BF), (F16, F16), (BF, F32)):
        dy, w = torch.ones(rows, k, dtype=dtype, device="cuda"), torch.zeros(k, n, dtype=dtype, device="cuda")
        w[0] = 3.0                                           # D = 3
        gate, up = torch.full((rows, n), 0.5, dtype=kept, device="cuda"), torch.full((rows, n), 2.0, dtype=kept, device="cuda")
        gate[:, 0], gate[:, 1], gate[:, 2], gate[:, n - 1] = -INF, INF, float("nan"), -INF
        dg, du = (torch.full((rows, n), 7.0, dtype=kept, device="cuda") for _ in range(2))
        L.ciera_glu_grad(dy, w, gate, up, dg, du, act=act)
        for c in (0, n - 1):
            assert (dg[:, c] == 0).all() and (du[:, c] == 0).all()
        assert (dg[:, 1] == 6).all() and (du[:, 1] == INF).all()
        assert torch.isnan(dg[:, 2]).all() and torch.isnan(du[:, 2]).all()
        assert torch.isfinite(dg[:, 3:]).all() and torch.isfinite(du[:, 3:]).all()
        # the same from sums that are not finite
        wg = torch.zeros(k, n, dtype=dtype, device="cuda")
        wg[0, 0], wg[0, 1], wg[0, 2], wg[0, n - 1] = -INF, INF, float("nan"), -INF
        h = torch.full((rows, n), 7.0, dtype=kept, device="cuda")
        L.ciera_glu_mm(dy, wg, w, h, act=act)
        assert (h[:, 0] == 0).all() and (h[:, n - 1] == 0).all()
        assert (h[:, 1] == INF).all() and torch.isnan(h[:, 2]).all() and (h[:, 3:n - 1] == 0).all()


@pytest.mark.parametrize("rows,n", PLACES)
def test_gate_kept_past_the_end_of_its_type(rows, n):
    """A finite sum below -65504 that is kept in fp16 becomes -inf: h and both gradients are 0."""
    k = 8
    x = torch.full((rows, k), 100.0, dtype=F16, device="cuda")
    wg, wu = torch.full((k, n), -1000.0, dtype=F16, device="cuda"), torch.full((k, n), 0.25, dtype=F16, device="cuda")
    h, gate, up, dg, du = (torch.full((rows, n), 7.0, dtype=F16, device="cuda") for _ in range(5))
    L.ciera_glu_mm(x, wg, wu, h, gate=gate, up=up)
    assert (h == 0).all() and (gate == -INF).all() and (up == 200).all()
    L.ciera_glu_grad(x, wu, gate, up, dg, du)
    assert (dg == 0).all() and (du == 0).all()
    dx = torch.full_like(x, 7.0)
    L.ciera_glu_xgrad(dg, du, wg, wu, dx, transpose_w=True)
    assert (dx == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,n", PLACES)
def test_large_gradients_of_closed_gates(rows, n, act):
    """D U is past the range of 32 bits, D U act'(G) is not."""
    k = 8
    dy, w = torch.zeros(rows, k, dtype=BF, device="cuda"), torch.zeros(1, k, n, dtype=BF, device="cuda")
    dy[:, 0], w[0, 0] = 1e20, 2.0
    gate = torch.full((rows, n), -2000.0, dtype=F32, device="cuda")
    gate[:, 1::3] = -2.0 if act == "gelu" else -30.0
    up = torch.full((rows, n), 3e18, dtype=F32, device="cuda")
    up[:, 0::3] = 1e25
    up[:, 2::3] = -3e38
    if act == "silu":
        up[:, 1::3] = 1e25
    dg, du = (torch.full((rows, n), 7.0, dtype=F32, device="cuda") for _ in range(2))
    L.ciera_glu_grad(dy, w[0], gate, up, dg, du, act=act)
    want = P.glu_grad(np64(dy), np64(w), np64(gate), np64(up), [0, rows], act)
    assert np.isfinite(want[0][0]).all() and np.abs(want[0][0]).max() < 3e38
    close(dg, *want[0], "dgate")
    close(du, *want[1], "dup")


# ----------------------------------------------------- large tiles, every type

# Aligned sizes that fill the card with tiles of 256 rows: the last column tile a part, stages of
# which the last is a part, one matrix, whole tiles only.
TILES = [(4300, 200, 2056, 14, 3), (4096, 72, 2304, 1, 0), (9000, 256, 2560, 2, 0), (8192, 64, 2048, 4, 0)]


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", TILES)
def test_large_tiles_of_every_type(shape, transpose, dtype, out):
    check_glu(shape, transpose, dtype, out, act="silu", keep=True)
    check_glu(shape, transpose, dtype, out, act="gelu", keep=False)
    check_grad(shape, transpose, dtype, out, act="silu")
    check_xgrad(shape, transpose, dtype, out)


# Rows that are not aligned, in groups long enough for tiles whatever the block, and in groups
# around the lengths from which on blocks of 32 and 128 take them.
@pytest.mark.parametrize("dtype,out,block,scales,zeros", [(BF, BF, 128, BF, True), (F16, F32, 32, F16, False),
                                                          (BF, F32, 64, F16, True), (F16, F16, 64, BF, False)])
@pytest.mark.parametrize("shape", [(8300, 201, 4100, 7, 3), (9001, 129, 2056, 1, 1), (5000, 77, 2056, 50, 0),
                                   (9800, 131, 1032, 50, 2), (9300, 63, 1032, 50, 0)])
def test_4_bit_products_of_rows_anywhere(shape, dtype, out, block, scales, zeros):
    check_gq(shape, dtype, out, block, scales, zeros)


# -------------------------------------------------------------- finding a workgroup's group

@pytest.mark.parametrize("groups", [1, 2, 63, 64, 65, 128, 192, 193, 255, 256, 257, 512, 513])
@pytest.mark.parametrize("most", [2, 40])
def test_groups_around_whole_waves_of_them(groups, most):
    """Offsets are looked at 64 or 256 groups at a time; some without rows, the first and last with."""
    say(f"[gpu] {groups} groups of up to {most} rows")
    rng = np.random.default_rng(groups * 100 + most)
    counts = rng.integers(0, most + 1, size=groups)
    counts[0] = counts[-1] = most
    if groups > 70:
        counts[5:70] = 0
    offsets = [0] + np.cumsum(counts).tolist()
    rows, k, n = offsets[-1], 24, 40
    x, w = rand((rows, k), BF, 1), rand((groups, k, n), BF, 2, 0.1)
    off = off_dev(offsets)
    want, err = P.sums(np64(x), np64(w), offsets)
    y, h = (torch.full((rows + 3, n), 7.0, dtype=BF, device="cuda") for _ in range(2))
    L.ciera_group_mm(x, w, y[:rows], offsets=off)
    close(y[:rows], want, err, "y")
    L.ciera_glu_mm(x, w, w, h[:rows], offsets=off)
    close(h[:rows], *P.gated(want, err, want, err, "silu"), "h")
    assert (y[rows:] == 7).all() and (h[rows:] == 7).all()
