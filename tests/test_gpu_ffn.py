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
