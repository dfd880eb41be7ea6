"""The gated feed-forward block, its backward pass and the 4-bit integer operators on the GPU
against the plain 64-bit forms of oracle/ffn_oracle.py."""
import numpy as np
import pytest
import torch

from oracle import ffn_oracle as P

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import lossless_weight_compression_amd as L  # noqa: E402
from lossless_weight_compression_amd.layer import GqMatrix, LayerCodec  # noqa: E402
from tests.gpu_harness import say  # noqa: E402

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}  # half a step, relative
KIND = {BF: "bf16", F16: "fp16"}


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def off_dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def close(got, want, err, what):
    """Each value within its error in 32 bits and one rounding."""
    tol = P.rounding(want, err, UNIT[got.dtype])
    off = np.abs(np64(got) - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off / tol):.3g} tolerances, first " \
                          f"{np.argwhere(bad)[:3].tolist()}"


def split(rows, groups, seed, tail=0):
    """Ascending offsets: uneven, empty groups among them, `tail` rows behind the last."""
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, rows - tail + 1, size=groups - 1)) if groups > 1 else np.zeros(0, int)
    if groups > 3:
        cuts[1] = cuts[0]
    return [0] + cuts.tolist() + [rows - tail]


def stack64(w, transpose):
    return np64(w).transpose(0, 2, 1) if transpose else np64(w)


def check_glu(shape, transpose, dtype, out, act="silu", keep=True, std=0.1):
    rows, k, n, groups, tail = shape
    say(f"[gpu] glu_mm {shape} transpose={transpose} {dtype} -> {out} {act} keep={keep}")
    ws = (groups, n, k) if transpose else (groups, k, n)
    x, wg, wu = rand((rows, k), dtype, 1), rand(ws, dtype, 2, std), rand(ws, dtype, 3, std)
    offsets = split(rows, groups, rows + k, tail)
    off = off_dev(offsets)
    res = [torch.full((rows, n), 7.0, dtype=out, device="cuda") for _ in range(3)]
    L.ciera_glu_mm(x, wg, wu, res[0], offsets=off, transpose_w=transpose, act=act,
                   gate=res[1] if keep else None, up=res[2] if keep else None)
    want = P.glu(np64(x), stack64(wg, transpose), stack64(wu, transpose), offsets, act)
    end = offsets[-1]
    for r, (v, e), what in list(zip(res, want, ("h", "gate", "up")))[:3 if keep else 1]:
        close(r[:end], v[:end], e[:end], what)
    for r in res:
        assert (r[end:] == 7.0).all()
    if not keep:
        assert (res[1] == 7.0).all() and (res[2] == 7.0).all()
    again = torch.full_like(res[0], 7.0)
    L.ciera_glu_mm(x, wg, wu, again, offsets=off, transpose_w=transpose, act=act)
    assert torch.equal(again, res[0])


def check_grad(shape, transpose, dtype, out, act="silu"):
    rows, k, n, groups, tail = shape
    say(f"[gpu] glu_grad {shape} transpose={transpose} {dtype} -> {out} {act}")
    dy = rand((rows, k), dtype, 1)
    w = rand((groups, n, k) if transpose else (groups, k, n), dtype, 2, 0.1)
    gate, up = rand((rows, n), out, 3, 2.0), rand((rows, n), out, 4)
    offsets = split(rows, groups, rows + k, tail)
    off = off_dev(offsets)
    dg, du = torch.full_like(gate, 7.0), torch.full_like(gate, 7.0)
    L.ciera_glu_grad(dy, w, gate, up, dg, du, offsets=off, transpose_w=transpose, act=act)
    end = offsets[-1]
    want = P.glu_grad(np64(dy), stack64(w, transpose), np64(gate), np64(up), offsets, act)
    for r, (v, e), what in zip((dg, du), want, ("dgate", "dup")):
        close(r[:end], v[:end], e[:end], what)
        assert (r[end:] == 7.0).all()
    again = [torch.full_like(gate, 7.0) for _ in range(2)]
    L.ciera_glu_grad(dy, w, gate, up, *again, offsets=off, transpose_w=transpose, act=act)
    assert torch.equal(again[0], dg) and torch.equal(again[1], du)


def check_xgrad(shape, transpose, dtype, out):
    rows, k, n, groups, tail = shape
    say(f"[gpu] glu_xgrad {shape} transpose={transpose} {dtype} -> {out}")
    dg, du = rand((rows, k), dtype, 1), rand((rows, k), dtype, 2)
    ws = (groups, n, k) if transpose else (groups, k, n)
    wg, wu = rand(ws, dtype, 3, 0.1), rand(ws, dtype, 4, 0.1)
    offsets = split(rows, groups, rows + k, tail)
    off = off_dev(offsets)
    dx = torch.full((rows, n), 7.0, dtype=out, device="cuda")
    L.ciera_glu_xgrad(dg, du, wg, wu, dx, offsets=off, transpose_w=transpose)
    v, e = P.glu_xgrad(np64(dg), np64(du), stack64(wg, transpose), stack64(wu, transpose), offsets)
    end = offsets[-1]
    close(dx[:end], v[:end], e[:end], "dx")
    assert (dx[end:] == 7.0).all()
    again = torch.full_like(dx, 7.0)
    L.ciera_glu_xgrad(dg, du, wg, wu, again, offsets=off, transpose_w=transpose)
    assert torch.equal(again, dx)


# rows, K, N, groups, rows behind the last group
SHAPES = [(1, 8, 8, 1, 0), (1, 2048, 64, 8, 0), (5, 1, 1, 3, 1), (7, 33, 17, 5, 2), (16, 64, 128, 2, 0),
          (40, 100, 36, 70, 3), (129, 130, 131, 4, 1), (300, 256, 256, 3, 9), (640, 96, 320, 2, 0),
          (97, 1447, 129, 6, 0), (260, 2048, 96, 300, 4), (1, 7168, 40, 1, 0), (512, 512, 512, 1, 0),
          (1111, 64, 264, 2, 5), (64, 7, 2048, 3, 0), (33, 1024, 1000, 2, 1)]
TYPES = [(BF, BF), (F16, F16), (BF, F32), (F16, F32)]


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_glu_mm(shape, transpose, dtype, out):
    check_glu(shape, transpose, dtype, out, act="gelu" if shape[0] % 2 else "silu", keep=shape[1] % 2 == 0 or out is F32)


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_glu_grad(shape, transpose, dtype, out):
    check_grad(shape, transpose, dtype, out, act="silu" if shape[0] % 2 else "gelu")


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_glu_xgrad(shape, transpose, dtype, out):
    check_xgrad(shape, transpose, dtype, out)


# Sizes that fill the card, aligned and nearly so, tile after tile; few rows to many groups.
LARGE = [(4300, 200, 2056, 14, 3), (4200, 8, 2048, 16, 0), (8500, 64, 1032, 33, 7), (4096, 72, 2304, 1, 0),
         (9001, 128, 1000, 5, 0), (6000, 328, 1544, 3, 1), (18000, 192, 520, 70, 11), (4300, 201, 2056, 14, 3),
         (4300, 200, 2051, 14, 3), (6000, 100, 777, 40, 2), (700, 1100, 136, 4, 2), (2200, 1447, 777, 13, 5),
         (9000, 256, 2560, 2, 0), (5000, 64, 4104, 2, 3), (200, 256, 1024, 150, 2), (200, 250, 1000, 150, 0),
         (90, 1064, 4096, 4, 1)]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F16, F32)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", LARGE)
def test_large(shape, transpose, dtype, out):
    check_glu(shape, transpose, dtype, out, act="silu", keep=dtype is BF)
    check_grad(shape, transpose, dtype, out, act="gelu")
    check_xgrad(shape, transpose, dtype, out)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_every_gate(act):
    """Pre-activations over the whole range: with one contraction step of 1 the gate's sum is the
    weight itself, with up 1 the result is the activation."""
    for dtype in (BF, F16):
        bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
        v = bits.view(dtype)
        v = v[torch.isfinite(v)]
        n = v.numel()
        x, one = torch.ones(1, 1, dtype=dtype, device="cuda"), torch.ones(1, 1, n, dtype=dtype, device="cuda")
        out = torch.empty(1, n, dtype=F32, device="cuda")
        L.ciera_glu_mm(x, v.reshape(1, 1, n), one, out, act=act)
        with np.errstate(over="ignore", invalid="ignore"):
            vv = np64(v)[None]
            want, err = P.act_value(vv, act)
            slope, eslope = P.act_slope(np.clip(vv, -1e6, 1e6), act)
        close(out, want, err + np.abs(vv) * 2.0 ** -126, f"{act} {dtype}")
        dg, du = torch.empty_like(out), torch.empty_like(out)
        L.ciera_glu_grad(x, one, v.reshape(1, n).float(), torch.ones_like(out), dg, du, act=act)
        close(dg, slope, eslope + 2.0 ** -120, f"slope {act} {dtype}")
        close(du, want, err + np.abs(vv) * 2.0 ** -126, f"value {act} {dtype}")


# ------------------------------------------------------------------------ 4-bit integers

def host(q):
    """Codes (one per value), scales in 32 bits and zeros of a GqMatrix."""
    codes = P.gq_unpack(q.codes.cpu().numpy().reshape(q.groups, q.rows, -1))
    return codes, q.scales.float().cpu().numpy(), None if q.zeros is None else q.zeros.cpu().numpy()


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("block,scales", [(32, BF), (64, F16), (128, BF), (128, F16)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 2048), (2, 31, 33), (3, 128, 64), (1, 129, 257), (5, 40, 100),
                                   (1, 700, 130), (2, 300, 515), (70, 3, 5), (1, 2048, 8)])
def test_quantize_and_back(shape, axis, dtype, block, scales, zeros):
    groups, rows, cols = shape
    say(f"[gpu] gq_quantize {shape} axis={axis} {dtype} {block} {scales} zeros={zeros}")
    x = rand(shape, F32, 7)
    x = (x * torch.exp2(torch.randint(-6, 7, (groups, rows, 1), device="cuda").float())).to(dtype)
    flat = x.view(-1)
    flat[: flat.numel() // 9] = flat[: flat.numel() // 9].abs()
    q = GqMatrix(*((rows, cols) if axis else (cols, rows)), groups=groups, block=block, dtype=scales, with_zeros=zeros)
    for t in (q.codes, q.scales) + ((q.zeros,) if zeros else ()):
        t.view(torch.uint8).fill_(0xa5)
    q.quantize(x, axis)
    codes, s, z = host(q)
    src = x if axis else x.transpose(1, 2)
    want = [P.gq_quantize(m.float().cpu().numpy(), block, KIND[scales], zeros) for m in src]
    assert np.array_equal(s, np.stack([w[1] for w in want]))
    if zeros:
        assert np.array_equal(z, np.stack([w[2] for w in want]))
    assert np.array_equal(codes, np.stack([w[0] for w in want]))
    vals, _ = P.gq_values(codes, s, z, block)
    for out in (BF, F16, F32):
        back = torch.full(src.shape, 7.0, dtype=out, device="cuda")
        q.dequantize(back)
        close(back, vals[..., :src.shape[2]], 0 * vals[..., :src.shape[2]], f"back {out}")
        exact = torch.from_numpy(vals[..., :src.shape[2]]).to(F32).to(out)
        assert torch.equal(back.cpu(), exact)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("zeros", [True, False])
def test_quantize_what_is_not_finite(zeros, axis, dtype):
    x = rand((1, 160, 160), dtype, 8)
    x[0, 3, 5], x[0, 40, 70], x[0, 150, 155] = float("inf"), float("nan"), float("-inf")
    x[0, 64:96, 64:96] = 0
    q = GqMatrix(160, 160, block=32, with_zeros=zeros).quantize(x, axis)
    codes, s, z = host(q)
    want = P.gq_quantize((x[0] if axis else x[0].t()).float().cpu().numpy(), 32, "bf16", zeros)
    assert np.array_equal(np.isnan(s[0]), np.isnan(want[1])) and np.isnan(s).sum() == 3
    assert np.array_equal(np.nan_to_num(s[0]), np.nan_to_num(want[1]))
    assert np.array_equal(codes[0], want[0]) and (z is None or np.array_equal(z[0], want[2]))
    back = q.dequantize()
    assert torch.isnan(back).sum() == 3 * 32 - 0
    assert (back[0, 64:96, 64:96] == 0).all()
    big = torch.full((1, 1, 4), 6e4 if dtype is F16 else 1e7, dtype=dtype, device="cuda")
    q = GqMatrix(1, 4, dtype=F16, with_zeros=zeros).quantize(big)
    assert torch.isnan(q.scales).all() == (dtype is not F16)


def make_gq(groups, rows, cols, block, scales, zeros, seed, std=0.1):
    w = rand((groups, rows, cols), F32, seed, std)
    return GqMatrix(rows, cols, groups=groups, block=block, dtype=scales, with_zeros=zeros).quantize(w)


def gq64(q):
    """Values and magnitudes in 64 bits."""
    codes, s, z = host(q)
    return P.gq_values(codes, s, z, q.block)


def check_gq(shape, dtype, out, block, scales, zeros, act="silu"):
    rows, k, n, groups, tail = shape
    say(f"[gpu] gq_mm {shape} {dtype} -> {out} block={block} {scales} zeros={zeros}")
    x = rand((rows, k), dtype, 11)
    w, w2 = (make_gq(groups, n, k, block, scales, zeros, 12 + i) for i in (0, 1))
    offsets = split(rows, groups, rows + k, tail)
    off, end = off_dev(offsets), offsets[-1]
    y, h = (torch.full((rows, n), 7.0, dtype=out, device="cuda") for _ in range(2))
    L.ciera_gq_mm(x, w, y, offsets=off)
    L.ciera_gq_glu(x, w, w2, h, offsets=off, act=act)
    g, eg = P.gq_sums(np64(x), *gq64(w), offsets, block)
    u, eu = P.gq_sums(np64(x), *gq64(w2), offsets, block)
    close(y[:end], g[:end], eg[:end], "y")
    hh, eh = P.gated(g, eg, u, eu, act)
    close(h[:end], hh[:end], eh[:end], "h")
    assert (y[end:] == 7.0).all() and (h[end:] == 7.0).all()
    y2, h2 = torch.full_like(y, 7.0), torch.full_like(h, 7.0)
    L.ciera_gq_mm(x, w, y2, offsets=off)
    L.ciera_gq_glu(x, w, w2, h2, offsets=off, act=act)
    assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype,out,block,scales", [(BF, BF, 128, BF), (F16, F16, 32, F16), (BF, F32, 64, F16),
                                                    (F16, F32, 128, BF), (BF, BF, 32, BF)])
@pytest.mark.parametrize("shape", SHAPES)
def test_gq_products(shape, dtype, out, block, scales, zeros):
    check_gq(shape, dtype, out, block, scales, zeros, act="gelu" if shape[0] % 2 else "silu")


GQ_LARGE = [(4300, 200, 520, 14, 3), (2000, 2048, 264, 3, 0), (3000, 640, 1000, 40, 2), (700, 1447, 777, 4, 2),
            (4096, 128, 1024, 1, 0), (200, 1024, 1024, 150, 2), (64, 2048, 4096, 1, 0), (9, 7168, 2048, 1, 0),
            (1025, 384, 130, 1, 1), (20, 2048, 2048, 8, 0), (600, 256, 520, 9, 1)]


@pytest.mark.parametrize("dtype,out,block,zeros", [(BF, BF, 128, True), (F16, F32, 32, False), (BF, F32, 64, True)])
@pytest.mark.parametrize("shape", GQ_LARGE)
def test_gq_products_large(shape, dtype, out, block, zeros):
    check_gq(shape, dtype, out, block, BF, zeros)


def test_gq_by_value():
    """Every code, zero and position: one-hot rows of x read the weights back exactly."""
    k, n = 256, 32
    for block in (32, 64, 128):
        for dtype in (BF, F16):
            rng = np.random.default_rng(9)
            codes = rng.integers(0, 16, size=(1, n, k)).astype(np.uint8)
            zeros = rng.integers(0, 16, size=(1, n, k // block)).astype(np.uint8)
            scales = torch.from_numpy(np.exp2(rng.integers(-6, 6, size=(1, n, k // block)))).to(BF).cuda()
            q = GqMatrix(n, k, block=block, codes=torch.from_numpy(P.gq_pack(codes)).cuda(), scales=scales,
                         zeros=torch.from_numpy(zeros).cuda())
            want = P.gq_values(codes, scales.float().cpu().numpy(), zeros, block)[0][0].T
            x = torch.eye(k, dtype=dtype, device="cuda")
            y = torch.empty(k, n, dtype=F32, device="cuda")
            L.ciera_gq_mm(x, q, y)
            assert np.array_equal(np64(y), want)
            # one token at a time
            for i in (0, 1, 31, 32, 127, 128, 255):
                y1 = torch.empty(1, n, dtype=F32, device="cuda")
                L.ciera_gq_mm(x[i:i + 1], q, y1)
                assert np.array_equal(np64(y1)[0], want[i])


# Sizes whose tiles of 128 rows fill the card.
@pytest.mark.parametrize("dtype,out,block,scales,zeros", [(BF, BF, 128, BF, True), (F16, F32, 32, F16, False),
                                                          (BF, F32, 64, F16, True), (F16, F16, 128, F16, False),
                                                          (BF, BF, 32, BF, True)])
@pytest.mark.parametrize("shape", [(9000, 200, 2056, 14, 3), (8200, 1447, 1000, 20, 0), (8192, 256, 4100, 3, 7)])
def test_gq_products_in_tiles(shape, dtype, out, block, scales, zeros):
    check_gq(shape, dtype, out, block, scales, zeros)


# Contractions longer than what is kept in LDS at a time (x, scales), and shorter than one stage.
@pytest.mark.parametrize("dtype,out,block,scales,zeros", [(BF, BF, 128, BF, True), (F16, F32, 32, F16, True),
                                                          (BF, F32, 64, F16, False), (F16, F16, 32, BF, False)])
@pytest.mark.parametrize("shape", [(9000, 1104, 2056, 14, 1), (9000, 40, 2056, 14, 0), (9000, 8, 2056, 14, 0),
                                   (700, 4400, 1100, 40, 1), (700, 4397, 300, 60, 0), (500, 2049, 1100, 40, 0)])
def test_gq_products_long_and_short(shape, dtype, out, block, scales, zeros):
    check_gq(shape, dtype, out, block, scales, zeros)


def inside(shape, dtype, seed, pad=(3, 5), std=1.0):
    """A matrix (or stack) in the middle of a larger buffer of other numbers, and the buffer."""
    wide = list(shape)
    wide[-1] += pad[1] * 2
    wide[-2] += pad[0] * 2
    buf = rand(wide, dtype, seed, std)
    cut = buf[..., pad[0]:pad[0] + shape[-2], pad[1]:pad[1] + shape[-1]]
    return cut, buf


@pytest.mark.parametrize("rows,k,n,pad", [(20, 72, 80, (1, 3)), (300, 200, 328, (2, 8)), (300, 201, 327, (2, 5)),
                                          (5000, 128, 1032, (3, 8)), (1, 264, 64, (0, 1))])
@pytest.mark.parametrize("transpose", [False, True])
def test_strides_and_neighbours(rows, k, n, pad, transpose):
    """Operands and results inside larger buffers: what lies around the results stays."""
    groups, offsets = 2, [0, rows // 3, rows]
    off = off_dev(offsets)
    ws = (groups, n, k) if transpose else (groups, k, n)
    x, _ = inside((rows, k), BF, 1, pad)
    (wg, _), (wu, _) = inside(ws, BF, 2, pad, 0.1), inside(ws, BF, 3, pad, 0.1)
    outs = [inside((rows, n), BF, 4 + i, pad) for i in range(3)]
    before = [b.clone() for _, b in outs]
    L.ciera_glu_mm(x, wg, wu, outs[0][0], offsets=off, transpose_w=transpose, gate=outs[1][0], up=outs[2][0])
    want = P.glu(np64(x), stack64(wg, transpose), stack64(wu, transpose), offsets, "silu")
    for (o, _), (v, e), what in zip(outs, want, ("h", "gate", "up")):
        close(o, v, e, what)
    (gate, _), (up, _) = inside((rows, n), BF, 7, pad), inside((rows, n), BF, 8, pad)
    dy, w = x, wg
    grads = [inside((rows, n), BF, 9 + i, pad) for i in range(2)]
    gbefore = [b.clone() for _, b in grads]
    L.ciera_glu_grad(dy, w, gate, up, grads[0][0], grads[1][0], offsets=off, transpose_w=transpose)
    want = P.glu_grad(np64(dy), stack64(w, transpose), np64(gate), np64(up), offsets, "silu")
    for (o, _), (v, e), what in zip(grads, want, ("dgate", "dup")):
        close(o, v, e, what)
    dx, dbuf = inside((rows, n), BF, 12, pad)
    dbefore = dbuf.clone()
    x2, _ = inside((rows, k), BF, 13, (pad[0], pad[1] + 1))          # another row stride than x's
    for second in (x2, x):
        L.ciera_glu_xgrad(x, second, wg, wu, dx, offsets=off, transpose_w=transpose)
        v, e = P.glu_xgrad(np64(x), np64(second), stack64(wg, transpose), stack64(wu, transpose), offsets)
        close(dx, v, e, "dx")
    q, q2 = make_gq(groups, n, k, 64, BF, True, 14), make_gq(groups, n, k, 64, BF, True, 15)
    y, ybuf = inside((rows, n), BF, 16, pad)
    ybefore = ybuf.clone()
    L.ciera_gq_mm(x, q, y, offsets=off)
    g, eg = P.gq_sums(np64(x), *gq64(q), offsets, 64)
    u, eu = P.gq_sums(np64(x), *gq64(q2), offsets, 64)
    close(y, g, eg, "gq")
    L.ciera_gq_glu(x, q, q2, y, offsets=off)
    close(y, *P.gated(g, eg, u, eu, "silu"), "gq glu")
    back, bbuf = inside((groups, n, k), F16, 17, pad)
    bbefore = bbuf.clone()
    q.dequantize(back)
    assert torch.equal(back, torch.from_numpy(gq64(q)[0][..., :k]).to(F32).to(F16).cuda())
    for buf, was in [(b, c) for (_, b), c in zip(outs + grads, before + gbefore)] + [(dbuf, dbefore), (ybuf, ybefore),
                                                                                     (bbuf, bbefore)]:
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[..., pad[0]:buf.shape[-2] - pad[0], pad[1]:buf.shape[-1] - pad[1]] = False
        assert torch.equal(buf[mask], was[mask])


@pytest.mark.parametrize("rows,n", [(9, 40), (300, 264), (300, 131), (5000, 1024)])
def test_columns_of_one_buffer(rows, n):
    """gate, up, dgate and dup side by side in one buffer; packed gate and up weights."""
    k, groups = 128, 2
    offsets = [0, rows // 2, rows]
    off = off_dev(offsets)
    x = rand((rows, k), BF, 1)
    packed = rand((groups, k, 2 * n), BF, 2, 0.1)
    wg, wu = packed[..., :n], packed[..., n:]
    buf = torch.zeros(rows, 5 * n, dtype=BF, device="cuda")
    h, gate, up, dgate, dup = (buf[:, i * n:(i + 1) * n] for i in range(5))
    L.ciera_glu_mm(x, wg, wu, h, offsets=off, gate=gate, up=up)
    want = P.glu(np64(x), np64(wg), np64(wu), offsets, "silu")
    for o, (v, e) in zip((h, gate, up), want):
        close(o, v, e, "forward")
    w = rand((groups, k, n), BF, 3, 0.1)
    L.ciera_glu_grad(x, w, gate, up, dgate, dup, offsets=off)
    for o, (v, e) in zip((dgate, dup), P.glu_grad(np64(x), np64(w), np64(gate), np64(up), offsets, "silu")):
        close(o, v, e, "backward")
    dx = torch.empty(rows, k, dtype=BF, device="cuda")
    L.ciera_glu_xgrad(dgate, dup, wg, wu, dx, offsets=off, transpose_w=True)
    close(dx, *P.glu_xgrad(np64(dgate), np64(dup), np64(wg).transpose(0, 2, 1), np64(wu).transpose(0, 2, 1), offsets), "dx")


def all_calls(rows, k, n, groups, off, x, wt, q, o):
    L.ciera_glu_mm(x, wt[0], wt[1], o["h"], offsets=off, gate=o["gate"], up=o["up"])
    L.ciera_glu_grad(o["dy"], wt[2], o["gate"], o["up"], o["dgate"], o["dup"], offsets=off, transpose_w=True)
    L.ciera_glu_xgrad(o["dgate"], o["dup"], wt[0], wt[1], o["dx"], offsets=off, transpose_w=True)
    L.ciera_gq_glu(x, q[0], q[1], o["qh"], offsets=off)
    L.ciera_gq_mm(o["qh"], q[2], o["qy"], offsets=off)
    q[3].quantize(wt[0], 0)
    q[3].dequantize(o["back"])


def operands(rows, k, n, groups, seed):
    x = rand((rows, k), BF, seed)
    wt = [rand((groups, k, n), BF, seed + 1, 0.05), rand((groups, k, n), BF, seed + 2, 0.05),
          rand((groups, n, k), BF, seed + 3, 0.05)]
    q = [make_gq(groups, n, k, 128, BF, True, seed + 4), make_gq(groups, n, k, 128, BF, True, seed + 5),
         make_gq(groups, k, n, 128, BF, True, seed + 6), GqMatrix(n, k, groups=groups)]
    o = {c: torch.zeros(rows, n, dtype=BF, device="cuda") for c in ("h", "gate", "up", "dgate", "dup", "qh")}
    o.update({c: torch.zeros(rows, k, dtype=BF, device="cuda") for c in ("dx", "qy")})
    o["dy"], o["back"] = rand((rows, k), BF, seed + 7), torch.zeros(groups, n, k, dtype=BF, device="cuda")
    return x, wt, q, o


GRAPHS = [(8, 256, 384, 4), (700, 256, 384, 2), (2600, 512, 2056, 2)]


@pytest.mark.parametrize("rows,k,n,groups", GRAPHS)
def test_captured_and_replayed(rows, k, n, groups):
    """Every call in one graph, replayed with new inputs and offsets, other work in between."""
    x, wt, q, o = operands(rows, k, n, groups, 21)
    off = off_dev(split(rows, groups, 1))
    all_calls(rows, k, n, groups, off, x, wt, q, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        all_calls(rows, k, n, groups, off, x, wt, q, o)
    for i in range(4):
        x.copy_(rand((rows, k), BF, 50 + i))
        o["dy"].copy_(rand((rows, k), BF, 60 + i))
        off.copy_(off_dev(split(rows, groups, 70 + i, tail=i)))
        for c in o:
            if c != "dy":
                o[c].fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = {c: t.clone() for c, t in o.items()}
        for c in o:
            if c != "dy":
                o[c].fill_(3.0)
        all_calls(rows, k, n, groups, off, x, wt, q, o)
        for c in o:
            assert torch.equal(got[c], o[c]), (i, c)
        assert torch.isfinite(got["dx"].float()).all()


@pytest.mark.parametrize("rows,k,n,groups", GRAPHS)
def test_on_side_streams_at_once(rows, k, n, groups):
    """The same work on two streams at once, neither of them the current one, equals each alone."""
    sets = [operands(rows, k, n, groups, 100 + 40 * i) for i in range(2)]
    offs = [off_dev(split(rows, groups, 5 + i)) for i in range(2)]
    alone = []
    for (x, wt, q, o), off in zip(sets, offs):
        all_calls(rows, k, n, groups, off, x, wt, q, o)
        torch.cuda.synchronize()
        alone.append({c: t.clone() for c, t in o.items()})
        for c in o:
            if c != "dy":
                o[c].fill_(3.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for (x, wt, q, o), off, s in zip(sets, offs, streams):
            with torch.cuda.stream(s):
                all_calls(rows, k, n, groups, off, x, wt, q, o)
    torch.cuda.synchronize()
    for (x, wt, q, o), was in zip(sets, alone):
        for c in o:
            assert torch.equal(o[c], was[c]), c


@pytest.mark.parametrize("rows,k,n", [(90, 64, 72), (3000, 520, 2056)])
@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 10, 2000, 60], [90, 60, 30, 0],
                                     [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1]])
def test_offsets_out_of_order_stay_inside(offsets, rows, k, n):
    """Results are unspecified then; buffers next to them stay as they were."""
    off = off_dev(offsets)
    x, wg, wu = rand((rows, k), BF, 1), rand((3, k, n), BF, 2, 0.1), rand((3, k, n), BF, 3, 0.1)
    wd = rand((3, n, k), BF, 4, 0.1)
    q, q2 = make_gq(3, n, k, 32, BF, True, 5), make_gq(3, n, k, 32, BF, True, 6)
    frames = {}

    def framed(name, cols):
        buf = torch.full((rows + 8, cols + 16), 5.0, dtype=BF, device="cuda")
        frames[name] = buf
        return buf[4:4 + rows, 8:8 + cols]

    h, gate, up, dg, du, y = (framed(c, n) for c in ("h", "gate", "up", "dg", "du", "y"))
    dx = framed("dx", k)
    L.ciera_glu_mm(x, wg, wu, h, offsets=off, gate=gate, up=up)
    L.ciera_glu_grad(x, wd, gate, up, dg, du, offsets=off, transpose_w=True)
    L.ciera_glu_xgrad(dg, du, wg, wu, dx, offsets=off, transpose_w=True)
    L.ciera_gq_mm(x, q, y, offsets=off)
    L.ciera_gq_glu(x, q, q2, y, offsets=off)
    torch.cuda.synchronize()
    for name, buf in frames.items():
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[4:4 + rows, 8:buf.shape[1] - 8] = False
        assert (buf[mask] == 5.0).all(), name


def test_one_group_without_offsets():
    for rows, k, n in ((1, 40, 24), (77, 129, 130), (700, 256, 264)):
        x, wg, wu = rand((rows, k), F16, 1), rand((k, n), F16, 2, 0.1), rand((k, n), F16, 3, 0.1)
        h, gate, up = (torch.empty(rows, n, dtype=F16, device="cuda") for _ in range(3))
        L.ciera_glu_mm(x, wg, wu, h, gate=gate, up=up, act="gelu")
        want = P.glu(np64(x), np64(wg)[None], np64(wu)[None], [0, rows], "gelu")
        for o, (v, e) in zip((h, gate, up), want):
            close(o, v, e, "forward")
        dg, du, dx = torch.empty_like(h), torch.empty_like(h), torch.empty_like(x)
        L.ciera_glu_grad(x, wg, gate, up, dg, du, act="gelu")
        for o, (v, e) in zip((dg, du), P.glu_grad(np64(x), np64(wg)[None], np64(gate), np64(up), [0, rows], "gelu")):
            close(o, v, e, "grad")
        L.ciera_glu_xgrad(dg, du, wg, wu, dx, transpose_w=True)
        close(dx, *P.glu_xgrad(np64(dg), np64(du), np64(wg).T[None], np64(wu).T[None], [0, rows]), "dx")
        q = make_gq(1, n, k, 64, F16, False, 4)
        L.ciera_gq_mm(x, q, h)
        close(h, *P.gq_sums(np64(x), *gq64(q), [0, rows], 64), "gq")


@pytest.mark.parametrize("rows", [3, 700])
def test_sizes_of_nothing(rows):
    """No contraction: sums of nothing; no rows in any group: nothing written."""
    off = off_dev([0, rows // 3, rows])
    x, w = torch.empty(rows, 0, dtype=BF, device="cuda"), torch.empty(2, 0, 40, dtype=BF, device="cuda")
    h, gate, up = (torch.full((rows, 40), 7.0, dtype=BF, device="cuda") for _ in range(3))
    L.ciera_glu_mm(x, w, w, h, offsets=off, gate=gate, up=up)
    assert (h == 0).all() and (gate == 0).all() and (up == 0).all()
    g = rand((rows, 40), BF, 1)
    L.ciera_glu_grad(x, w, g, g, gate.fill_(7.0), up.fill_(7.0), offsets=off)
    assert (gate == 0).all() and (up == 0).all()
    L.ciera_glu_xgrad(x, x, w, w, h.fill_(7.0), offsets=off)
    assert (h == 0).all()
    q = GqMatrix(40, 0, groups=2)
    L.ciera_gq_mm(x, q, h.fill_(7.0), offsets=off)
    assert (h == 0).all()
    none = off_dev([0, 0, 0])
    x, w = rand((rows, 64), BF, 2), rand((2, 64, 40), BF, 3)
    q = make_gq(2, 40, 64, 32, BF, True, 4)
    for call in (lambda: L.ciera_glu_mm(x, w, w, h, offsets=none, gate=gate, up=up),
                 lambda: L.ciera_glu_grad(x, w, g, g, gate, up, offsets=none),
                 lambda: L.ciera_glu_xgrad(x, x, w, w, h, offsets=none),
                 lambda: L.ciera_gq_mm(x, q, h, offsets=none), lambda: L.ciera_gq_glu(x, q, q, h, offsets=none)):
        for t in (h, gate, up):
            t.fill_(7.0)
        call()
        assert (h == 7).all() and (gate == 7).all() and (up == 7).all()


@pytest.mark.parametrize("rows,k,n", [(9, 64, 64), (300, 128, 264), (300, 129, 70), (5000, 64, 1032)])
def test_what_is_not_finite_stays_in_its_row(rows, k, n):
    x = rand((rows, k), BF, 1)
    bad = [2, rows // 2, rows - 1]
    x[bad[0], 3], x[bad[1], k - 1], x[bad[2], 5] = float("inf"), float("nan"), float("-inf")
    off = off_dev([0, rows // 3, rows])
    wg, wu = rand((2, k, n), BF, 2, 0.1), rand((2, k, n), BF, 3, 0.1)
    q = make_gq(2, n, k, 64, BF, True, 4)
    good = torch.ones(rows, dtype=torch.bool, device="cuda")
    good[bad] = False
    clean = torch.where(torch.isfinite(x.float()), x, torch.zeros_like(x))
    h, h0 = (torch.empty(rows, n, dtype=BF, device="cuda") for _ in range(2))
    for call in (lambda x, o: L.ciera_glu_mm(x, wg, wu, o, offsets=off), lambda x, o: L.ciera_gq_mm(x, q, o, offsets=off),
                 lambda x, o: L.ciera_gq_glu(x, q, q, o, offsets=off),
                 lambda x, o: L.ciera_glu_xgrad(x, x, wg, wu, o, offsets=off)):
        call(x, h)
        call(clean, h0)
        assert torch.equal(h[good], h0[good]) and torch.isfinite(h0.float()).all()
        assert not torch.isfinite(h[bad[1]].float()).any()
    L.ciera_gq_mm(x, q, h, offsets=off)
    assert torch.isnan(h[bad].float()).all()
    # a NaN scale spoils its column, nothing else
    q.scales[0, 1, 0] = float("nan")
    q.scales[1, 1, 0] = float("nan")
    L.ciera_gq_mm(clean, q, h, offsets=off)
    assert torch.isnan(h[:, 1].float()).all() and torch.isfinite(torch.cat((h[:, :1], h[:, 2:]), 1).float()).all()


def test_strides_of_zero():
    """One matrix for all groups, one row for all rows."""
    k, n, rows = 96, 72, 50
    off = off_dev([0, 10, 10, 50])
    w = rand((k, n), BF, 1, 0.1)
    ws = w.expand(3, k, n)
    x = rand((1, k), BF, 2).expand(rows, k)
    h = torch.empty(rows, n, dtype=BF, device="cuda")
    L.ciera_glu_mm(x, ws, ws, h, offsets=off)
    one = torch.empty(1, n, dtype=BF, device="cuda")
    L.ciera_glu_mm(x[:1], w, w, one)
    want = P.glu(np64(x), np64(ws), np64(ws), [0, 10, 10, 50], "silu")[0]
    close(h, *want, "h")
    close(one, want[0][:1], want[1][:1], "one")
    q = GqMatrix(k, n, groups=1, block=32).quantize(x.new_zeros(1, n).expand(k, n))
    assert (q.dequantize() == 0).all()


@pytest.mark.parametrize("groups", [65, 257, 3000])
def test_many_groups(groups):
    rng = np.random.default_rng(groups)
    counts = rng.integers(0, 3, size=groups)
    counts[groups // 2] = 70
    offsets = [0] + np.cumsum(counts).tolist()
    rows, k, n = offsets[-1], 40, 24
    x = rand((rows, k), BF, 1)
    wg, wu = rand((groups, k, n), BF, 2, 0.1), rand((groups, k, n), BF, 3, 0.1)
    off = off_dev(offsets)
    h, gate, up = (torch.empty(rows, n, dtype=BF, device="cuda") for _ in range(3))
    L.ciera_glu_mm(x, wg, wu, h, offsets=off, gate=gate, up=up)
    for o, (v, e) in zip((h, gate, up), P.glu(np64(x), np64(wg), np64(wu), offsets, "silu")):
        close(o, v, e, "forward")
    dx = torch.empty(rows, k, dtype=BF, device="cuda")
    L.ciera_glu_xgrad(gate, up, wg, wu, dx, offsets=off, transpose_w=True)
    close(dx, *P.glu_xgrad(np64(gate), np64(up), np64(wg).transpose(0, 2, 1), np64(wu).transpose(0, 2, 1), offsets), "dx")
    q = make_gq(groups, n, k, 32, BF, True, 4)
    L.ciera_gq_mm(x, q, h, offsets=off)
    close(h, *P.gq_sums(np64(x), *gq64(q), offsets, 32), "gq")


def test_far_ends_of_large_operands():
    """Elements past 2^31 bytes and 2^31 elements: the last group of a large stack, rows far apart."""
    groups, k, n = 17, 16384, 8192
    wg = torch.zeros(groups, k, n, dtype=BF, device="cuda")         # 4.6 GB
    wg[-1, -64:, -64:] = rand((64, 64), BF, 1, 0.1)
    x = torch.zeros(4, k, dtype=BF, device="cuda")
    x[:, -64:] = rand((4, 64), BF, 2)
    off = off_dev([0] * groups + [4])
    h, gate, up = (torch.empty(4, n, dtype=BF, device="cuda") for _ in range(3))
    L.ciera_glu_mm(x, wg, wg, h, offsets=off, gate=gate, up=up)
    want = np64(x[:, -64:]) @ np64(wg[-1, -64:, -64:])
    assert np.abs(np64(gate)[:, -64:] - want).max() < 0.02 and torch.equal(gate, up)
    assert (h[:, :-64] == 0).all()
    q = GqMatrix(n, k, groups=groups, block=128)
    q.quantize(wg, 0)                                               # 1.1 GB of codes
    del wg
    y = torch.empty(4, n, dtype=BF, device="cuda")
    L.ciera_gq_mm(x, q, y, offsets=off)
    last = GqMatrix(n, k, block=128, codes=q.codes[-1:].clone(), scales=q.scales[-1:].clone(), zeros=q.zeros[-1:].clone())
    y2 = torch.empty_like(y)
    L.ciera_gq_mm(x, last, y2)
    assert torch.equal(y, y2) and y[:, -64:].abs().sum() > 0 and (y[:, :-64] == 0).all()
    far = torch.zeros(3, 1 << 30, dtype=BF, device="cuda")          # rows 2 GB apart
    view = far[:, :k]
    view.copy_(x[:3])
    L.ciera_gq_mm(view, last, y2[:3])
    assert torch.equal(y2[:3], y[:3])


def test_layer_from_streams_through_the_block():
    """A decoded layer's gate, up and down matrices: forward and backward on the full weights, and
    a token on 4-bit copies of them, as they would be used."""
    h, f, e, world, tokens, top = 256, 128, 4, 2, 37, 2
    shapes = [(h, f)] * e + [(h, f)] * e + [(f, h)] * e
    codec = LayerCodec(shapes, BF, world)
    full = [rand(s, BF, 300 + i, 0.05) for i, s in enumerate(shapes)]
    codec.seed_cache(full)
    new = [w + rand(w.shape, BF, 400 + i, 0.01) for i, w in enumerate(full)]
    for r in range(world):
        flat = [w.reshape(-1) for w in new]
        codec.encode(r, [flat[i][codec.shard(i, r)[0]:sum(codec.shard(i, r))].clone() for i in range(len(shapes))])
    assert int(codec.decode().item()) == 0
    wg, wu, wd = codec.stack(range(e)), codec.stack(range(e, 2 * e)), codec.stack(range(2 * e, 3 * e))
    assert torch.equal(wg, torch.stack(new[:e]))
    rng = np.random.default_rng(8)
    expert = np.concatenate([rng.permutation(e)[:top] for _ in range(tokens)])
    order = np.argsort(expert, kind="stable")
    token = torch.from_numpy(np.repeat(np.arange(tokens), top)[order]).cuda()
    offsets = [0] + np.cumsum(np.bincount(expert, minlength=e)).tolist()
    rows, off = len(order), off_dev([0] + np.cumsum(np.bincount(expert, minlength=e)).tolist())
    x = rand((tokens, h), BF, 500)[token]
    hid, gate, up, dg, du = (torch.empty(rows, f, dtype=BF, device="cuda") for _ in range(5))
    y, dx, dy = torch.empty_like(x), torch.empty_like(x), rand((rows, h), BF, 501)
    L.ciera_glu_mm(x, wg, wu, hid, offsets=off, gate=gate, up=up)
    L.ciera_group_mm(hid, wd, y, offsets=off)
    L.ciera_glu_grad(dy, wd, gate, up, dg, du, offsets=off, transpose_w=True)
    L.ciera_glu_xgrad(dg, du, wg, wu, dx, offsets=off, transpose_w=True)
    dwg, dwu, dwd = (torch.empty(w.shape, dtype=F32, device="cuda") for w in (wg, wu, wd))
    L.ciera_group_wgrad(x, dg, dwg, offsets=off)
    L.ciera_group_wgrad(x, du, dwu, offsets=off)
    L.ciera_group_wgrad(hid, dy, dwd, offsets=off)

    # against automatic differentiation in 64 bits on the CPU; each of up to four roundings to bf16
    # on the way to a gradient is off by 2^-8 of its size at most
    p = [t.detach().double().cpu().requires_grad_() for t in (x, wg, wu, wd)]
    parts = []
    for g in range(e):
        a, b = offsets[g], offsets[g + 1]
        z = p[0][a:b] @ p[1][g]
        parts.append((z * torch.sigmoid(z) * (p[0][a:b] @ p[2][g])) @ p[3][g])
    want = torch.cat(parts)
    (want * dy.double().cpu()).sum().backward()
    for got, ref, steps in ((y, want.detach(), 2), (dx, p[0].grad, 3), (dwg, p[1].grad, 3), (dwu, p[2].grad, 3),
                            (dwd, p[3].grad, 2)):
        assert float((got.double().cpu() - ref).norm() / ref.norm()) < steps * 2.0 ** -8

    # the same layer in 4 bits: what the copies stand for, multiplied in 64 bits
    for zeros in (True, False):
        qg, qu = (codec.quantize_groups(range(i * e, (i + 1) * e), zeros=zeros) for i in (0, 1))
        qd = codec.quantize_groups(range(2 * e, 3 * e), zeros=zeros)
        assert (qg.rows, qg.cols, qd.rows, qd.cols) == (f, h, h, f)
        off8 = [max(abs(float((q.dequantize().transpose(1, 2).double() - w.double()).norm() / w.double().norm())), 0)
                for q, w in ((qg, wg), (qu, wu), (qd, wd))]
        assert max(off8) < 0.15                          # 16 levels over about 5 deviations
        L.ciera_gq_glu(x, qg, qu, hid, offsets=off)
        L.ciera_gq_mm(hid, qd, y, offsets=off)
        g, eg = P.gq_sums(np64(x), *gq64(qg), offsets, 128)
        u, eu = P.gq_sums(np64(x), *gq64(qu), offsets, 128)
        close(hid, *P.gated(g, eg, u, eu, "silu"), "hidden")
        close(y, *P.gq_sums(np64(hid), *gq64(qd), offsets, 128), "output")


def test_gradients_against_differences():
    """dx, dW_gate and dW_up of sum(dy (h w_down)) by central differences of the kernels' own
    forward pass in fp32 results."""
    rows, k, n, groups = 6, 16, 8, 2
    offsets = [0, 2, 6]
    off = off_dev(offsets)
    x, wg, wu = rand((rows, k), F16, 1), rand((groups, k, n), F16, 2, 0.3), rand((groups, k, n), F16, 3, 0.3)
    wd, dy = rand((groups, n, k), F16, 4, 0.3), rand((rows, k), F16, 5)
    for act in ("silu", "gelu"):
        h, gate, up = (torch.empty(rows, n, dtype=F32, device="cuda") for _ in range(3))

        def loss(x, wg, wu):
            L.ciera_glu_mm(x, wg, wu, h, offsets=off, act=act)
            return sum(float((h[a:b].double() @ wd[g].double() * dy[a:b].double()).sum())
                       for g, (a, b) in enumerate(zip(offsets, offsets[1:])))

        L.ciera_glu_mm(x, wg, wu, torch.empty_like(h), offsets=off, gate=gate, up=up, act=act)
        dg, du = torch.empty_like(h), torch.empty_like(h)
        L.ciera_glu_grad(dy, wd, gate, up, dg, du, offsets=off, transpose_w=True, act=act)
        dx = torch.empty(rows, k, dtype=F32, device="cuda")
        L.ciera_glu_xgrad(dg.half(), du.half(), wg, wu, dx, offsets=off, transpose_w=True)
        dw = [torch.empty(groups, k, n, dtype=F32, device="cuda") for _ in range(2)]
        for d, t in zip(dw, (dg, du)):
            L.ciera_group_wgrad(x, t.half(), d, offsets=off)
        rng = np.random.default_rng(6)
        for i, (t, d) in enumerate(((x, dx), (wg, dw[0]), (wu, dw[1]))):
            for _ in range(12):
                at = tuple(int(rng.integers(0, s)) for s in t.shape)
                step = 2.0 ** -5
                v = [[x, wg, wu], [x, wg, wu]]
                for s, side in ((-1, 0), (1, 1)):
                    moved = t.clone()
                    moved[at] += s * step
                    v[side][i] = moved
                width = float(v[1][i][at].double() - v[0][i][at].double())
                slope = (loss(*v[1]) - loss(*v[0])) / width
                # third derivatives times the step squared, roundings of dg and du to fp16
                assert abs(slope - float(d[at])) < 0.02 * max(1.0, abs(slope))
