"""The products grouped by expert, their gradients and the 4-bit operators on
the GPU against the plain 64-bit forms of oracle/ops_oracle.py."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import lossless_weight_compression_amd as L  # noqa: E402
from lossless_weight_compression_amd.layer import LayerCodec, MxMatrix  # noqa: E402
from tests.gpu_harness import say  # noqa: E402

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}  # half a step, relative


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, device="cuda", generator=gen(seed)) * std).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def off_dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def close(got, want, mag, steps, dtype, what):
    err = np.abs(np64(got) - want)
    tol = P.tolerance(want, mag, steps, UNIT[dtype])
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.3g} tolerances, first " \
                          f"{np.argwhere(bad)[:3].tolist()}"


def split(rows, groups, seed, tail=0):
    """Ascending offsets: uneven, empty groups among them, `tail` rows behind the last."""
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, rows - tail + 1, size=groups - 1)) if groups > 1 else np.zeros(0, int)
    if groups > 3:
        cuts[1] = cuts[0]
    return [0] + cuts.tolist() + [rows - tail]


# rows, K, N, groups, rows behind the last group
SHAPES = [(1, 8, 8, 1, 0), (1, 2048, 64, 8, 0), (5, 1, 1, 3, 1), (7, 33, 17, 5, 2), (16, 64, 128, 2, 0),
          (40, 100, 36, 70, 3), (129, 130, 131, 4, 1), (300, 256, 256, 3, 9), (640, 96, 320, 2, 0),
          (97, 1447, 129, 6, 0), (260, 2048, 96, 300, 4), (1, 7168, 40, 1, 0), (512, 512, 512, 1, 0),
          (1111, 64, 264, 2, 5), (64, 7, 2048, 3, 0), (33, 1024, 1000, 2, 1)]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F16), (BF, F32), (F16, F32)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_group_mm(shape, transpose, dtype, out):
    rows, k, n, groups, tail = shape
    say(f"[gpu] group_mm {shape} transpose={transpose} {dtype} -> {out}")
    x = rand((rows, k), dtype, 1)
    w = rand((groups, n, k) if transpose else (groups, k, n), dtype, 2, 0.1)
    offsets = split(rows, groups, rows + k, tail)
    y = torch.full((rows, n), 7.0, dtype=out, device="cuda")
    L.ciera_group_mm(x, w, y, offsets=off_dev(offsets), transpose_w=transpose)
    w64 = np64(w).transpose(0, 2, 1) if transpose else np64(w)
    want, mag = P.group_mm(np64(x), w64, offsets, np.full((rows, n), 7.0))
    close(y, want, mag, k, out, "y")
    assert (y[offsets[-1]:] == 7.0).all()
    again = torch.full_like(y, 7.0)
    L.ciera_group_mm(x, w, again, offsets=off_dev(offsets), transpose_w=transpose)
    assert torch.equal(y, again)


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F16), (BF, F32), (F16, F32)])
@pytest.mark.parametrize("shape", SHAPES)
def test_group_wgrad(shape, dtype, out):
    rows, k, n, groups, tail = shape
    say(f"[gpu] group_wgrad {shape} {dtype} -> {out}")
    x, dy = rand((rows, k), dtype, 3), rand((rows, n), dtype, 4, 0.1)
    offsets = split(rows, groups, rows + n, tail)
    g = torch.full((groups, k, n), 7.0, dtype=out, device="cuda")
    L.ciera_group_wgrad(x, dy, g, offsets=off_dev(offsets))
    want, mag = P.group_wgrad(np64(x), np64(dy), offsets)
    close(g, want, mag, rows, out, "dw")
    again = torch.full_like(g, 5.0)
    L.ciera_group_wgrad(x, dy, again, offsets=off_dev(offsets))
    assert torch.equal(g, again)


# Sizes that fill the card: many rows to a group (256 x 256 tiles read straight into LDS)
# and what only nearly qualifies.  rows, K, N, groups, rows behind the last group
LARGE = [(4300, 200, 2056, 14, 3), (4200, 8, 2048, 16, 0), (8500, 64, 1032, 33, 7), (4096, 72, 2304, 1, 0),
         (9001, 128, 1000, 5, 0), (8200, 136, 1024, 32, 100), (6000, 328, 1544, 3, 1), (18000, 40, 520, 70, 11),
         (4300, 201, 2056, 14, 3), (4300, 200, 2051, 14, 3), (6000, 100, 777, 40, 2), (700, 1100, 136, 4, 2),
         (520, 576, 300, 2, 0), (2200, 1447, 777, 13, 5)]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F32)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", LARGE)
def test_group_mm_large(shape, transpose, dtype, out):
    test_group_mm(shape, transpose, dtype, out)


# rows, K, N, groups, rows behind the last group: gradients of K x N
LARGE_GRADS = [(700, 1032, 1288, 8, 3), (3, 2056, 2048, 3, 0), (900, 264, 256, 70, 0), (5000, 1024, 520, 12, 9),
               (64, 4104, 2048, 1, 0), (1300, 776, 1000, 11, 1), (130, 520, 264, 300, 2), (1300, 777, 1001, 11, 1),
               (2006, 515, 777, 7, 9), (1500, 130, 64, 5, 0), (300, 100, 130, 1, 0)]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F32)])
@pytest.mark.parametrize("shape", LARGE_GRADS)
def test_group_wgrad_large(shape, dtype, out):
    test_group_wgrad(shape, dtype, out)


@pytest.mark.parametrize("one", [0, 5, 63, 64, 199])
def test_group_wgrad_all_rows_in_one_group(one):
    """All the work in one of many groups, the others' gradients zeros."""
    say(f"[gpu] wgrad, all rows in group {one}")
    groups = 64 if one < 64 else 200
    x, dy = rand((3000, 264), BF, 3), rand((3000, 512), BF, 4, 0.1)
    offsets = [0] * (one + 1) + [3000] * (groups - one)
    g = torch.full((groups, 264, 512), 7.0, dtype=F32, device="cuda")
    L.ciera_group_wgrad(x, dy, g, offsets=off_dev(offsets))
    want, mag = P.group_wgrad(np64(x), np64(dy), offsets)
    close(g, want, mag, 3000, F32, "dw")


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shape", LARGE)
def test_mx_mm_large(shape, out):
    test_mx_mm(shape, out)


@pytest.mark.parametrize("rows,k,n,groups", [(4300, 200, 2056, 14), (9001, 72, 1032, 5)])
def test_large_strides_and_neighbours(rows, k, n, groups):
    """Large tiles out of and into parts of larger buffers: nothing around the output
    changes, NaN around the operands and in rows of no group reach no result, infinities stay
    in their rows."""
    say(f"[gpu] large tiles, strides rows={rows} k={k} n={n}")
    nan = float("nan")
    offsets = split(rows, groups, 9, tail=30)
    off = off_dev(offsets)
    big_x = torch.full((rows + 2, k + 24), nan, dtype=BF, device="cuda")
    x = big_x[1:-1, 8:8 + k]
    x[:rows - 30] = rand((rows - 30, k), BF, 8)
    big_w = torch.full((groups, k + 3, n + 16), nan, dtype=BF, device="cuda")
    w = big_w[:, 1:k + 1, 8:8 + n]
    w.copy_(rand((groups, k, n), BF, 9))
    big_y = torch.full((rows + 2, n + 19), 7.0, dtype=BF, device="cuda")
    y = big_y[1:-1, 5:5 + n]
    ok = slice(0, rows - 30)
    want, mag = P.group_mm(np64(x), np64(w), offsets, np.full((rows, n), 7.0))
    L.ciera_group_mm(x, w, y, offsets=off)
    close(y[ok], want[ok], mag[ok], k, BF, "y")
    y[ok] = 7.0
    assert (big_y == 7.0).all()
    wt = torch.full((groups, n + 1, k + 16), nan, dtype=BF, device="cuda")[:, 1:, 8:8 + k]
    wt.copy_(w.transpose(1, 2))
    L.ciera_group_mm(x, wt, y, offsets=off, transpose_w=True)
    close(y[ok], want[ok], mag[ok], k, BF, "y, [N, K]")
    y[ok] = 7.0
    assert (big_y == 7.0).all()
    x[100, 3], x[700, 0] = float("inf"), nan
    L.ciera_group_mm(x, w, y, offsets=off)
    assert (~torch.isfinite(y)).any(1).nonzero().flatten().tolist() == [100, 700]
    x[100, 3], x[700, 0] = 1.0, 1.0
    # gradients of [n, k] matrices, in larger ones
    big_dy = torch.full((rows, n + 8), nan, dtype=BF, device="cuda")
    dy = big_dy[:, 8:]
    dy[ok] = rand((rows - 30, n), BF, 10)
    big_g = torch.full((groups, n + 2, k + 5), 7.0, dtype=F32, device="cuda")
    g = big_g[:, 1:-1, 3:3 + k]
    L.ciera_group_wgrad(dy, x, g, offsets=off)
    want, mag = P.group_wgrad(np64(dy), np64(x), offsets)
    close(g, want, mag, rows, F32, "dw")
    g.fill_(7.0)
    assert (big_g == 7.0).all()


@pytest.mark.parametrize("rows", [3, 24, 700])
def test_sizes_of_nothing(rows):
    say(f"[gpu] K = 0, empty groups, rows={rows}")
    y = torch.full((rows, 40), 7.0, dtype=BF, device="cuda")
    off = off_dev([0, rows // 3, rows - 1])
    for tr in (False, True):
        y.fill_(7.0)
        w = torch.zeros((2, 40, 0) if tr else (2, 0, 40), dtype=BF, device="cuda")
        L.ciera_group_mm(torch.zeros(rows, 0, dtype=BF, device="cuda"), w, y, offsets=off, transpose_w=tr)
        assert (y[:-1] == 0).all() and (y[-1] == 7).all()
    a, b = MxMatrix(rows, 0), MxMatrix(40, 0, groups=2)
    y.fill_(7.0)
    L.ciera_mx_mm(a, b, y, offsets=off)
    assert (y[:-1] == 0).all() and (y[-1] == 7).all()
    # no row in any group: gradients are zero, products leave everything
    x, none = rand((rows, 48), BF, 5), off_dev([0, 0, 0])
    g = torch.full((2, 48, 40), 7.0, dtype=BF, device="cuda")
    L.ciera_group_wgrad(x, rand((rows, 40), BF, 6), g, offsets=none)
    assert (g == 0).all()
    g.fill_(7.0)
    L.ciera_group_wgrad(x[:0], rand((0, 40), BF, 6), g, offsets=none)
    assert (g == 0).all()
    y.fill_(7.0)
    L.ciera_group_mm(x, rand((2, 48, 40), BF, 7), y, offsets=none)
    assert (y == 7).all()


@pytest.mark.parametrize("rows,k,n", [(40, 72, 80), (300, 200, 328), (300, 201, 327)])
def test_strides_and_neighbours(rows, k, n):
    """Operands and outputs that are parts of larger buffers: column slices (rows that
    start anywhere), one matrix for every group, values around the output untouched,
    NaN in the neighbours never read into a result."""
    say(f"[gpu] strides rows={rows} k={k} n={n}")
    nan = float("nan")
    for dtype in (BF, F16):
        for shift in (1, 8):
            big_x = torch.full((rows + 2, k + 19), nan, dtype=dtype, device="cuda")
            x = big_x[1:-1, shift:shift + k]
            x.copy_(rand((rows, k), dtype, 8))
            big_w = torch.full((3, k + 3, n + 11), nan, dtype=dtype, device="cuda")
            w = big_w[:, 1:k + 1, shift:shift + n]
            w.copy_(rand((3, k, n), dtype, 9))
            offsets = [0, rows // 4, rows // 4, rows - 3]
            x[rows - 3:] = nan
            big_y = torch.full((rows + 2, n + 21), 7.0, dtype=dtype, device="cuda")
            y = big_y[1:-1, shift + 1:shift + 1 + n]
            L.ciera_group_mm(x, w, y, offsets=off_dev(offsets))
            want, mag = P.group_mm(np64(x), np64(w), offsets, np.full((rows, n), 7.0))
            ok = slice(0, rows - 3)
            close(y[ok], want[ok], mag[ok], k, dtype, "y")
            y.fill_(7.0)
            assert (big_y == 7.0).all()
            # the same weights for every group, as a stack of stride 0
            one = w[1][None].expand(3, k, n)
            L.ciera_group_mm(x, one, y, offsets=off_dev(offsets))
            want, mag = P.group_mm(np64(x), np64(one), offsets, np.full((rows, n), 7.0))
            close(y[ok], want[ok], mag[ok], k, dtype, "y, one matrix")
            dy = rand((rows, n + 5), dtype, 10)[:, 5:]
            big_g = torch.full((3, k + 1, n + 7), 7.0, dtype=dtype, device="cuda")
            g = big_g[:, :k, shift:shift + n] if shift < 7 else big_g[:, :k, 7:]
            g = g[:, :, :n]
            L.ciera_group_wgrad(x, dy, g, offsets=off_dev(offsets))
            want, mag = P.group_wgrad(np64(x), np64(dy), offsets)
            close(g, want, mag, rows, dtype, "dw")
            g.fill_(7.0)
            assert (big_g == 7.0).all()


@pytest.mark.parametrize("groups", [65, 3000])
def test_many_groups(groups):
    """More groups than a wave adds up at once, most of them empty or of one row."""
    say(f"[gpu] {groups} groups")
    rows, k, n = groups + 900, 40, 24
    offsets = split(rows, groups, 3, tail=2)
    off = off_dev(offsets)
    x, w, dy = rand((rows, k), BF, 24), rand((groups, k, n), BF, 25), rand((rows, n), BF, 26)
    y = torch.full((rows, n), 7.0, dtype=BF, device="cuda")
    L.ciera_group_mm(x, w, y, offsets=off)
    want, mag = P.group_mm(np64(x), np64(w), offsets, np.full((rows, n), 7.0))
    close(y, want, mag, k, BF, "y")
    g = torch.full((groups, k, n), 7.0, dtype=BF, device="cuda")
    L.ciera_group_wgrad(x, dy, g, offsets=off)
    want, mag = P.group_wgrad(np64(x), np64(dy), offsets)
    close(g, want, mag, rows, BF, "dw")
    qx, qw = MxMatrix(rows, k).quantize(x), MxMatrix(n, k, groups=groups).quantize(w, axis=0)
    y.fill_(7.0)
    L.ciera_mx_mm(qx, qw, y, offsets=off)
    want, mag = P.group_mm(mx64(qx)[0], mx64(qw).transpose(0, 2, 1), offsets, np.full((rows, n), 7.0))
    close(y, want, mag, k, BF, "4-bit y")


def test_one_row_for_all():
    """x and dy as one row repeated (stride 0), and every operand the same memory."""
    say("[gpu] broadcast rows")
    for rows in (40, 700, 5000):
        x, dy = rand((1, 256), BF, 27).expand(rows, 256), rand((1, 264), BF, 28).expand(rows, 264)
        w, offsets = rand((2, 256, 2056), BF, 29), [0, rows // 3, rows]
        y = torch.zeros(rows, 2056, dtype=BF, device="cuda")
        L.ciera_group_mm(x, w, y, offsets=off_dev(offsets))
        want, mag = P.group_mm(np64(x), np64(w), offsets, np.zeros((rows, 2056)))
        close(y, want, mag, 256, BF, "y")
        g = torch.zeros(2, 256, 264, dtype=F32, device="cuda")
        L.ciera_group_wgrad(x, dy, g, offsets=off_dev(offsets))
        want, mag = P.group_wgrad(np64(x), np64(dy), offsets)
        close(g, want, mag, rows, F32, "dw")
    s = rand((256, 256), BF, 30)
    y = torch.zeros(256, 256, dtype=F32, device="cuda")
    L.ciera_group_mm(s, s, y, transpose_w=True)
    want, mag = P.group_mm(np64(s), np64(s).T[None], [0, 256], np.zeros((256, 256)))
    close(y, want, mag, 256, F32, "s s^T")


@pytest.mark.parametrize("rows,k,n", [(9, 64, 64), (300, 128, 264), (300, 129, 70)])
def test_infinities_stay_in_their_rows(rows, k, n):
    say(f"[gpu] infinities rows={rows} k={k} n={n}")
    x, w = rand((rows, k), BF, 11), rand((2, k, n), BF, 12)
    x[2, 5], x[4, 0] = float("inf"), float("nan")
    offsets = [0, 4, rows]
    y = torch.zeros(rows, n, dtype=BF, device="cuda")
    L.ciera_group_mm(x, w, y, offsets=off_dev(offsets))
    r = torch.zeros(rows, dtype=torch.bool)
    r[2] = r[4] = True
    assert torch.equal((~torch.isfinite(y)).any(1).cpu(), r) and torch.isnan(y[4]).all()
    assert torch.equal(torch.isinf(y[2]), w[0, 5] != 0)
    g = torch.zeros(2, k, n, dtype=BF, device="cuda")
    L.ciera_group_wgrad(x, rand((rows, n), BF, 13), g, offsets=off_dev(offsets))
    bad = (~torch.isfinite(g)).any(2).cpu()
    assert bad[0].nonzero().tolist() == [[5]] and bad[1].nonzero().tolist() == [[0]]


@pytest.mark.parametrize("rows,k,n", [(90, 64, 72), (3000, 520, 3080)])
@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 10, 2000, 60], [90, 60, 30, 0], [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1]])
def test_offsets_out_of_order_stay_inside(offsets, rows, k, n):
    """Unspecified rows, but nothing outside the operands is touched."""
    say(f"[gpu] offsets {offsets} rows={rows}")
    x, w = rand((rows, k), BF, 14), rand((3, k, n), BF, 15)
    buf = torch.full((rows + 200, n), 7.0, dtype=BF, device="cuda")
    L.ciera_group_mm(x, w, buf[100:100 + rows], offsets=off_dev(offsets))
    g = torch.full((5, k, n), 7.0, dtype=BF, device="cuda")
    L.ciera_group_wgrad(x, rand((rows, n), BF, 16), g[1:4], offsets=off_dev(offsets))
    qx, qw = MxMatrix(rows, k).quantize(x), MxMatrix(n, k, groups=3).quantize(w, axis=0)
    buf2 = torch.full((rows + 200, n), 7.0, dtype=BF, device="cuda")
    L.ciera_mx_mm(qx, qw, buf2[100:100 + rows], offsets=off_dev(offsets))
    torch.cuda.synchronize()
    for b in (buf, buf2):
        assert (b[:100] == 7).all() and (b[100 + rows:] == 7).all()
    assert (g[0] == 7).all() and (g[4] == 7).all() and torch.isfinite(g).all()


# ------------------------------------------------------------ 4-bit operators

def check_quantised(x, axis, q, what):
    x64 = np64(x)
    for g in range(x64.shape[0]):
        m = x64[g].T if axis == 0 else x64[g]
        codes, scales = P.mx_quantize(m)
        got_c, got_s = P.mx_unpack(q.codes[g].cpu().numpy()), q.scales[g].cpu().numpy()
        assert np.array_equal(got_s, scales), f"{what}: scales of {g} differ"
        assert np.array_equal(got_c, codes), f"{what}: codes of {g} differ at {np.argwhere(got_c != codes)[:4].tolist()}"


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 2048), (2, 31, 33), (3, 128, 64), (1, 129, 257), (5, 40, 100),
                                   (1, 1000, 8), (2, 300, 519), (1, 1, 129), (1, 513, 1), (4, 256, 384)])
def test_quantize_and_back(shape, axis, dtype):
    say(f"[gpu] quantize {shape} axis={axis} {dtype}")
    x = rand(shape, dtype, 20, 0.02)
    x = (x.float() * torch.exp2(torch.randint(-6, 7, shape, device="cuda", generator=gen(21)).float())).to(dtype)
    if x.numel() > 600:
        flat = x.view(-1)
        flat[100:200] = 0
        flat[::7] = torch.sign(flat[::7]) * 0.25    # many exact ties with powers of two around
        flat[3::11] = -0.0
    g, r, c = shape
    q = MxMatrix(c, r, groups=g) if axis == 0 else MxMatrix(r, c, groups=g)
    q.codes.fill_(0xEE)
    q.scales.fill_(0xEE)
    q.quantize(x, axis)
    check_quantised(x, axis, q, "q")
    # rows that start anywhere
    big = torch.zeros(g, r + 1, c + 5, dtype=dtype, device="cuda")
    big[:, 1:, 3:3 + c] = x
    p = MxMatrix(q.rows, q.cols, groups=g).quantize(big[:, 1:, 3:3 + c], axis)
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    for out in (BF, F16, F32):
        v = torch.stack([torch.from_numpy(P.mx_values(P.mx_unpack(q.codes[i].cpu().numpy()), q.scales[i].cpu().numpy())
                                          [:, :q.cols]) for i in range(g)]).to(out)
        buf = torch.full((g, q.rows + 1, q.cols + 3), 7.0, dtype=out, device="cuda")
        q.dequantize(buf[:, 1:, 2:2 + q.cols])
        assert torch.equal(buf[:, 1:, 2:2 + q.cols].cpu(), v)
        buf[:, 1:, 2:2 + q.cols] = 7.0
        assert (buf == 7).all()
        assert torch.equal(q.dequantize(torch.empty(g, q.rows, q.cols, dtype=out, device="cuda")).cpu(), v)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("axis", [0, 1])
def test_quantize_every_magnitude(dtype, axis):
    """Blocks around every power of two of the type, its subnormals, its largest value,
    infinities, NaN of either sign, negative zeros."""
    say(f"[gpu] quantize every magnitude axis={axis} {dtype}")
    if dtype == F32:
        exps = torch.arange(-149, 128, dtype=torch.float64)
    else:
        exps = torch.arange(-133, 128, dtype=torch.float64) if dtype == BF else torch.arange(-24, 16, dtype=torch.float64)
    m = torch.randn(len(exps), 128, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    x = (m.clamp(-1.99, 1.99) * torch.exp2(exps)[:, None]).to(dtype)
    big = torch.finfo(dtype).max
    extra = torch.zeros(12, 128, dtype=dtype)
    extra[0, :] = big
    extra[1, 5] = -big
    extra[2, 40], extra[3, 41] = float("inf"), float("-inf")
    extra[4, 99] = float("nan")
    extra[5, 127] = -torch.tensor(float("nan"))
    extra[6, :] = -0.0
    extra[7, 0], extra[7, 1] = torch.finfo(dtype).smallest_normal, -torch.finfo(dtype).smallest_normal / 2
    extra[8, ::2] = -1.0
    extra[9, :40] = torch.tensor([6, -6, 5, -5, 7, -7, 3.5, 2.5, .25, -.25] * 4, dtype=dtype)
    extra[10, 3] = torch.nextafter(torch.tensor(big, dtype=dtype).float(), torch.tensor(0.0)).to(dtype)
    x = torch.cat((x, extra))[None].cuda()
    xs = x.transpose(1, 2).contiguous() if axis == 0 else x
    q = MxMatrix(x.shape[1], 128).quantize(xs, axis)
    check_quantised(xs, axis, q, "q")
    v = q.dequantize(torch.empty(x.shape, dtype=F32, device="cuda"))
    n = len(exps)
    assert torch.isnan(v[0, n + 2, 32:64]).all() and torch.isnan(v[0, n + 4, 96:]).all()
    assert torch.isfinite(v[0, :n]).all() and torch.isnan(q.dequantize(torch.empty(x.shape, dtype=F16, device="cuda"))[0, n + 5, 96:]).all()


def mx_random(rows, cols, groups, seed):
    q = MxMatrix(rows, cols, groups=groups)
    kp = q.codes.shape[-1] * 2
    codes = torch.randint(0, 256, q.codes.shape, device="cuda", generator=gen(seed), dtype=torch.uint8)
    if kp != cols:  # codes past cols are zero
        mask = torch.zeros(kp, dtype=torch.uint8, device="cuda")
        mask[:cols] = 15
        codes &= mask[0::2] | (mask[1::2] << 4)
    q.codes.copy_(codes)
    q.scales.copy_(torch.randint(118, 128, q.scales.shape, device="cuda", generator=gen(seed + 1), dtype=torch.uint8))
    return q


def mx64(q):
    return P.mx_values(P.mx_unpack(q.codes.cpu().numpy()), q.scales.cpu().numpy())


@pytest.mark.parametrize("out", [BF, F16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_mx_mm(shape, out):
    rows, k, n, groups, tail = shape
    say(f"[gpu] mx_mm {shape} -> {out}")
    a, b = mx_random(rows, k, 1, 30), mx_random(n, k, groups, 32)
    offsets = split(rows, groups, rows + k, tail)
    y = torch.full((rows, n), 7.0, dtype=out, device="cuda")
    L.ciera_mx_mm(a, b, y, offsets=off_dev(offsets))
    want, mag = P.group_mm(mx64(a)[0], mx64(b).transpose(0, 2, 1), offsets, np.full((rows, n), 7.0))
    close(y, want, mag, k, out, "y")
    assert (y[offsets[-1]:] == 7.0).all()
    buf = torch.full((rows + 1, n + 3), 7.0, dtype=out, device="cuda")  # rows that start anywhere
    L.ciera_mx_mm(a, b, buf[1:, 1:n + 1], offsets=off_dev(offsets))
    assert torch.equal(buf[1:, 1:n + 1], y)
    buf[1:, 1:n + 1] = 7.0
    assert (buf == 7).all()


@pytest.mark.parametrize("rows", [4, 300])
def test_mx_mm_nan_scale(rows):
    say(f"[gpu] mx_mm NaN scales rows={rows}")
    x, w = rand((rows, 300), BF, 40), rand((200, 300), BF, 41)
    x[1, 200] = float("inf")
    w[7, 0] = float("nan")
    a, b = MxMatrix(rows, 300).quantize(x), MxMatrix(200, 300).quantize(w)
    y = torch.zeros(rows, 200, dtype=BF, device="cuda")
    L.ciera_mx_mm(a, b, y)
    want = torch.zeros(rows, 200, dtype=torch.bool)
    want[1], want[:, 7] = True, True
    assert torch.equal(torch.isnan(y).cpu(), want)


# ---------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("rows,k,n", [(300, 512, 256), (6000, 512, 2048)])
def test_on_a_side_stream(rows, k, n):
    """Every call on a stream other than the current one, beside a call of the same
    kind on the current one: each sees its own operands only."""
    say(f"[gpu] side stream rows={rows}")
    offsets = [0, rows // 3, rows // 3, rows - 10]
    off = off_dev(offsets)
    side = torch.cuda.Stream()
    res = {}
    for name in ("main", "side", "again"):
        seed = 50 if name != "side" else 60
        x, w, dy = rand((rows, k), BF, seed), rand((3, k, n), BF, seed + 1), rand((rows, n), BF, seed + 2)
        res[name] = dict(x=x, w=w, dy=dy, y=torch.zeros(rows, n, dtype=BF, device="cuda"),
                         g=torch.zeros(3, k, n, dtype=F32, device="cuda"), y4=torch.zeros(rows, n, dtype=BF, device="cuda"),
                         qx=MxMatrix(rows, k), qw=MxMatrix(n, k, groups=3))
    torch.cuda.synchronize()

    def go(r, stream):
        L.ciera_group_mm(r["x"], r["w"], r["y"], offsets=off, stream=stream)
        L.ciera_group_wgrad(r["x"], r["dy"], r["g"], offsets=off, stream=stream)
        r["qx"].quantize(r["x"], stream=stream)
        r["qw"].quantize(r["w"], axis=0, stream=stream)
        L.ciera_mx_mm(r["qx"], r["qw"], r["y4"], offsets=off, stream=stream)

    go(res["main"], None)
    go(res["side"], side)
    torch.cuda.synchronize()
    go(res["again"], None)
    torch.cuda.synchronize()
    for key in ("y", "g", "y4"):
        assert torch.equal(res["main"][key], res["again"][key]) and not torch.equal(res["main"][key], res["side"][key])
    want, mag = P.group_mm(np64(res["side"]["x"]), np64(res["side"]["w"]), offsets, np.zeros((rows, n)))
    close(res["side"]["y"], want, mag, k, BF, "y on the side stream")


@pytest.mark.parametrize("rows,k,n", [(8, 256, 384), (700, 256, 384), (2600, 1024, 3080)])
def test_captured_and_replayed(rows, k, n):
    """A step of a layer (products, gradients, quantisation, 4-bit product) captured
    once; each replay sees the inputs and offsets of its time and equals the eager calls."""
    say(f"[gpu] graph rows={rows}")
    groups = 5
    x, w, dy = rand((rows, k), BF, 70), rand((groups, k, n), BF, 71, 0.1), rand((rows, n), BF, 72)
    off = off_dev(split(rows, groups, 1))
    outs = [torch.zeros(rows, n, dtype=BF, device="cuda"), torch.zeros(rows, k, dtype=BF, device="cuda"),
            torch.zeros(groups, k, n, dtype=F32, device="cuda"), torch.zeros(rows, n, dtype=F16, device="cuda")]
    qx, qw = MxMatrix(rows, k), MxMatrix(n, k, groups=groups)

    def step():
        L.ciera_group_mm(x, w, outs[0], offsets=off)
        L.ciera_group_mm(dy, w, outs[1], offsets=off, transpose_w=True)
        L.ciera_group_wgrad(x, dy, outs[2], offsets=off)
        qx.quantize(x)
        qw.quantize(w, axis=0)
        L.ciera_mx_mm(qx, qw, outs[3], offsets=off)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(rand((rows, k), BF, 80 + i))
        dy.copy_(rand((rows, n), BF, 90 + i))
        off.copy_(off_dev(split(rows, groups, 2 + i, tail=i)))
        for o in outs:
            o.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.fill_(3.0)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


# -------------------------------------------------------- used together

def test_layer_from_streams_to_products():
    """A layer of experts encoded, decoded, viewed as stacks, applied to routed
    tokens, differentiated and quantised: as a training step uses them."""
    say("[gpu] decode -> stack -> products -> 4 bits")
    groups, dm, dff, rows = 6, 256, 192, 500
    shapes = [s for _ in range(groups) for s in ((dm, dff), (dm, dff), (dff, dm))]
    codec = LayerCodec(shapes, BF, 2, 512, "cuda", 10_000)
    ws = [rand(s, BF, 100 + i, 0.05) for i, s in enumerate(shapes)]
    codec.seed_cache(ws)
    for r in range(2):
        shards = []
        for i in range(len(shapes)):
            o, cnt = codec.shard(i, r)
            shards.append(ws[i].reshape(-1)[o:o + cnt].clone())
        codec.encode(r, shards)
    assert int(codec.decode().item()) == 0
    gate, up, down = (codec.stack(range(j, 3 * groups, 3)) for j in range(3))
    assert torch.equal(gate, torch.stack(ws[0::3])) and torch.equal(down, torch.stack(ws[2::3]))
    offsets = split(rows, groups, 5, tail=6)
    off = off_dev(offsets)
    x, dy = rand((rows, dm), BF, 130), rand((rows, dm), BF, 131)
    new = lambda c, dt=BF: torch.zeros(rows, c, dtype=dt, device="cuda")  # noqa: E731
    h1, h3, y = new(dff), new(dff), new(dm)
    L.ciera_group_mm(x, gate, h1, offsets=off)
    L.ciera_group_mm(x, up, h3, offsets=off)
    a = (torch.nn.functional.silu(h1.float()) * h3.float()).to(BF)
    L.ciera_group_mm(a, down, y, offsets=off)
    da, dx = new(dff), new(dm)
    L.ciera_group_mm(dy, down, da, offsets=off, transpose_w=True)
    dgate = torch.zeros(groups, dm, dff, dtype=F32, device="cuda")
    ddown = torch.zeros(groups, dff, dm, dtype=F32, device="cuda")
    L.ciera_group_wgrad(a, dy, ddown, offsets=off)
    L.ciera_group_mm(h3, gate, dx, offsets=off, transpose_w=True)
    L.ciera_group_wgrad(x, da, dgate, offsets=off)
    z = lambda c: np.zeros((rows, c))  # noqa: E731
    tr = lambda t: np64(t).transpose(0, 2, 1)  # noqa: E731
    for got, (p, q, k, c) in ((h1, (x, np64(gate), dm, dff)), (h3, (x, np64(up), dm, dff)), (y, (a, np64(down), dff, dm)),
                              (da, (dy, tr(down), dm, dff)), (dx, (h3, tr(gate), dff, dm))):
        want, mag = P.group_mm(np64(p), q, offsets, z(c))
        close(got, want, mag, k, BF, "product")
    for got, p, q in ((ddown, a, dy), (dgate, x, da)):
        want, mag = P.group_wgrad(np64(p), np64(q), offsets)
        close(got, want, mag, rows, F32, "gradient")
    # the 4-bit copy of the same weights and its product
    qg = codec.quantize(range(0, 3 * groups, 3), axis=0)
    check_quantised(gate, 0, qg, "gate")
    check_quantised(down, 1, codec.quantize(range(2, 3 * groups, 3), axis=1), "down, along the rows")
    again = MxMatrix(dff, dm, groups=groups)
    assert codec.quantize(range(0, 3 * groups, 3), into=again) is again and torch.equal(again.codes, qg.codes)
    gap = torch.zeros(groups, dm + 1, dff, dtype=BF, device="cuda")[:, 1:]  # matrices with gaps between them
    MxMatrix(dm, dff, groups=groups).quantize(gate).dequantize(gap)
    assert torch.equal(gap, MxMatrix(dm, dff, groups=groups).quantize(gate.contiguous()).dequantize())
    qx = MxMatrix(rows, dm).quantize(x)
    y4 = new(dff)
    L.ciera_mx_mm(qx, qg, y4, offsets=off)
    want, mag = P.group_mm(mx64(qx)[0], mx64(qg).transpose(0, 2, 1), offsets, z(dff))
    close(y4, want, mag, dm, BF, "4-bit product")
    for bad in ([], [0, 2], [0, 3, 9], [3, 0]):
        with pytest.raises(ValueError):
            codec.stack(bad)


def test_gradients_against_differences():
    """d/dw and d/dx of sum(dy * y) against central differences of the forward product
    (fp16 operands and steps that it holds exactly, fp32 results: the product is linear in each)."""
    say("[gpu] gradients against differences")
    rows, k, n, groups = 37, 24, 40, 3
    offsets = [0, 11, 11, 37]
    off = off_dev(offsets)
    q = lambda s, seed: torch.randint(-8, 9, s, device="cuda", generator=gen(seed)).half() / 8  # noqa: E731
    x, w, dy = q((rows, k), 140), q((groups, k, n), 141), q((rows, n), 142)

    def loss(x, w):
        y = torch.zeros(rows, n, dtype=F32, device="cuda")
        L.ciera_group_mm(x, w, y, offsets=off)
        return (y.double() * dy.double()).sum().item()

    dw = torch.zeros(groups, k, n, dtype=F32, device="cuda")
    dx = torch.zeros(rows, k, dtype=F32, device="cuda")
    L.ciera_group_wgrad(x, dy, dw, offsets=off)
    L.ciera_group_mm(dy, w, dx, offsets=off, transpose_w=True)
    rng = np.random.default_rng(4)
    for _ in range(12):
        g, a, b, i = (int(rng.integers(v)) for v in (groups, k, n, rows))
        wp, wm, xp, xm = w.clone(), w.clone(), x.clone(), x.clone()
        wp[g, a, b] += 0.5
        wm[g, a, b] -= 0.5
        xp[i, a] += 0.5
        xm[i, a] -= 0.5
        # all values are multiples of 2^-6 below 2^10: every sum is exact
        assert loss(x, wp) - loss(x, wm) == dw[g, a, b].item()
        assert loss(xp, w) - loss(xm, w) == dx[i, a].item()


def test_far_ends_of_large_operands():
    """Element offsets beyond 2^32 in the weights, the output and the 4-bit codes."""
    say("[gpu] offsets beyond 2^32")
    groups, k, n = 3, 64, 64
    w = torch.zeros(2 * (2 ** 31 + 4096) + k * n, dtype=BF, device="cuda")
    ws = torch.as_strided(w, (groups, k, n), (2 ** 31 + 4096, n, 1))
    ws.copy_(rand((groups, k, n), BF, 150))
    x = rand((40, k), BF, 151)
    off = off_dev([0, 10, 20, 40])
    y = torch.zeros(40, n, dtype=BF, device="cuda")
    L.ciera_group_mm(x, ws, y, offsets=off)
    want, mag = P.group_mm(np64(x), np64(ws), [0, 10, 20, 40], np.zeros((40, n)))
    close(y, want, mag, k, BF, "y")
    ld = 2 ** 27  # rows of an output 2^27 apart: row 39 lies past 2^32 elements
    big = torch.zeros(39 * ld + n, dtype=BF, device="cuda")
    yb = torch.as_strided(big, (40, n), (ld, 1))
    L.ciera_group_mm(x, ws, yb, offsets=off)
    assert torch.equal(yb, y)
    g = torch.as_strided(w, (groups, k, n), (2 ** 31 + 4096, n, 1))
    L.ciera_group_wgrad(x, y.clone(), g, offsets=off)
    want, mag = P.group_wgrad(np64(x), np64(y), [0, 10, 20, 40])
    close(g, want, mag, 40, BF, "dw")
    qs = MxMatrix(n, k, groups=groups).quantize(g, axis=0)
    check_quantised(g, 0, qs, "far")


def test_offsets_next_to_the_output():
    """Offsets that end where the output begins, or begin where it ends, are taken."""
    say("[gpu] offsets next to the output")
    rows, k, n, groups = 40, 64, 96, 3
    offsets = split(rows, groups, 5, tail=2)
    x, w = rand((rows, k), BF, 51), rand((groups, k, n), BF, 52, 0.1)
    want, mag = P.group_mm(np64(x), np64(w), offsets, np.full((rows, n), 7.0))
    size = rows * n
    buf = torch.full((size + 16,), 7.0, dtype=BF, device="cuda")
    y = buf[8:8 + size].view(rows, n)
    for off in (buf[:8].view(torch.int32), buf[8 + size:].view(torch.int32)):
        y.fill_(7.0)
        off.copy_(off_dev(offsets))
        L.ciera_group_mm(x, w, y, offsets=off)
        close(y, want, mag, k, BF, "y")
        assert off.tolist() == offsets
    with pytest.raises(L.CieraError):
        L.ciera_group_mm(x, w, y, offsets=buf[6:14].view(torch.int32))


@pytest.mark.parametrize("raw", [False, True])
def test_results_made_on_a_side_stream(raw):
    """Outputs that a call on another stream makes itself do not take memory that work
    still under way on the current one writes."""
    say(f"[gpu] results made on a side stream, raw handle {raw}")
    groups, r, c = 3, 256, 512
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    codec = LayerCodec([(r, c)] * groups, BF, 1, 512, "cuda", 10_000)
    for i in range(groups):
        codec.out_view(i).copy_(rand((r * c,), BF, 60 + i))
    want_q = codec.quantize(range(groups))
    want = want_q.dequantize()
    a = rand((4096, 4096), BF, 63)
    b = torch.empty_like(a)
    torch.cuda.synchronize()

    def under_way(shape, dtype):
        gone = torch.empty(shape, dtype=dtype, device="cuda")
        for _ in range(20):
            torch.mm(a, a, out=b)
        gone.fill_(7)

    under_way(want.shape, want.dtype)
    got = want_q.dequantize(stream=stream)
    under_way(want_q.codes.shape, torch.uint8)
    under_way(want_q.scales.shape, torch.uint8)
    got_q = codec.quantize(range(groups), stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(got_q.codes, want_q.codes) and torch.equal(got_q.scales, want_q.scales)
    codec.quantize(range(groups), stream=0)                # the default stream's handle
    assert torch.equal(want_q.dequantize(stream=0), want)


# Several tiles one after another to each workgroup of the large kernels, most of them whole,
# with several stages each, so that the next tile's loads and the last one's stores are under
# way together.  504 tiles: no half ones at the end; 360: the last ones halved; 481: whole and
# ragged ones in turn.  rows, K, N, groups, rows behind the last group
ROUNDS = [(9000, 584, 3584, 2, 3), (9000, 584, 2560, 2, 0), (9000, 328, 3080, 3, 1)]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F32)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", ROUNDS)
def test_group_mm_tile_after_tile(shape, transpose, dtype, out):
    test_group_mm(shape, transpose, dtype, out)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shape", ROUNDS + [(9000, 1447, 2560, 2, 0)])
def test_mx_mm_tile_after_tile(shape, out):
    test_mx_mm(shape, out)


# gradients of K x N: 512, 560 (more groups than a wave has lanes) and 480 tiles
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F32)])
@pytest.mark.parametrize("shape", [(2100, 2048, 2048, 8, 5), (9000, 512, 1024, 70, 0), (1500, 1288, 2560, 8, 1)])
def test_group_wgrad_tile_after_tile(shape, dtype, out):
    test_group_wgrad(shape, dtype, out)


# A few rows to each of many groups: 128 columns to a workgroup, whole and ragged ones; one
# step of the contraction to a wave, several, and ends inside one
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F16), (BF, F32), (F16, F32)])
@pytest.mark.parametrize("shape", [(200, 256, 1024, 150, 2), (200, 250, 1000, 150, 0), (190, 1064, 1024, 150, 1),
                                   (170, 777, 1160, 140, 0)])
def test_group_mm_few_rows_many_groups(shape, dtype, out):
    test_group_mm(shape, False, dtype, out)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("hot", [0, 77, 255])
def test_one_popular_group(hot, transpose):
    """Nearly all rows in one of many groups."""
    say(f"[gpu] popular group {hot} transpose={transpose}")
    rows, k, n, groups = 1500, 200, 520, 256
    counts = [1 if g % 5 == 0 else 0 for g in range(groups)]
    counts[hot] += rows - sum(counts)
    offsets = [0] + np.cumsum(counts).tolist()
    x, w = rand((rows, k), BF, 71), rand((groups, n, k) if transpose else (groups, k, n), BF, 72, 0.1)
    y = torch.full((rows, n), 7.0, dtype=BF, device="cuda")
    L.ciera_group_mm(x, w, y, offsets=off_dev(offsets), transpose_w=transpose)
    want, mag = P.group_mm(np64(x), np64(w).transpose(0, 2, 1) if transpose else np64(w), offsets, np.zeros((rows, n)))
    close(y, want, mag, k, BF, "y")
    qx, qw = MxMatrix(rows, k).quantize(x), MxMatrix(n, k, groups=groups).quantize(w, axis=1 if transpose else 0)
    L.ciera_mx_mm(qx, qw, y, offsets=off_dev(offsets))
    want, mag = P.group_mm(mx64(qx)[0], mx64(qw).transpose(0, 2, 1), offsets, np.zeros((rows, n)))
    close(y, want, mag, k, BF, "4-bit y")
    dy = rand((rows, n), BF, 73, 0.1)
    g = torch.full((groups, k, n), 7.0, dtype=F32, device="cuda")
    L.ciera_group_wgrad(x, dy, g, offsets=off_dev(offsets))
    want, mag = P.group_wgrad(np64(x), np64(dy), offsets)
    close(g, want, mag, rows, F32, "dw")


@pytest.mark.parametrize("dtype", [F16, F32])
def test_stacks_of_other_types(dtype):
    """fp16 and fp32 layers as stacks: equal distances, 4-bit copies, and products of
    those that the products take."""
    say(f"[gpu] stack and quantize of {dtype}")
    groups, dm, dff, rows = 4, 96, 131, 70
    codec = LayerCodec([s for _ in range(groups) for s in ((dm, dff), (dff, dm))], dtype, 1, 512, "cuda", 10_000)
    ws = [rand((dm, dff) if i % 2 == 0 else (dff, dm), dtype, 80 + i, 0.05) for i in range(2 * groups)]
    codec.seed_cache(ws)
    codec.encode(0, [w.reshape(-1) for w in ws])
    assert int(codec.decode().item()) == 0
    up, down = codec.stack(range(0, 2 * groups, 2)), codec.stack(range(1, 2 * groups, 2))
    assert up.dtype == dtype and torch.equal(up, torch.stack(ws[0::2])) and torch.equal(down, torch.stack(ws[1::2]))
    check_quantised(up, 0, codec.quantize(range(0, 2 * groups, 2), axis=0), "up, down the columns")
    check_quantised(down, 1, codec.quantize(range(1, 2 * groups, 2), axis=1), "down, along the rows")
    off = split(rows, groups, 5)
    x, y = rand((rows, dm), dtype, 90), torch.zeros(rows, dff, dtype=dtype, device="cuda")
    if dtype == F32:
        with pytest.raises(L.CieraError):
            L.ciera_group_mm(x, up, y, offsets=off_dev(off))
        return
    L.ciera_group_mm(x, up, y, offsets=off_dev(off))
    want, mag = P.group_mm(np64(x), np64(up), off, np.zeros((rows, dff)))
    close(y, want, mag, dm, dtype, "y")
