"""What the gated block and the 4-bit integer operators refuse, before any device call (fake
addresses, CPU tensors)."""
import ctypes

import pytest
import torch

L = pytest.importorskip("lossless_weight_compression_amd")
BF, F32, F16 = L.CIERA_BF16, L.CIERA_FP32, L.CIERA_FP16


def mat(at, rows, cols, dtype=BF, groups=1, ld=None, gs=None):
    ld = cols if ld is None else ld
    return L.Matrix(at, dtype, groups, rows, cols, ld, rows * ld if gs is None else gs)


def refused(code, call, *args, **kw):
    with pytest.raises(L.CieraError) as e:
        call(*args, stream=0, **kw)
    assert e.value.code == code


A, B, C, D, E, F, OFF = (0x1000000 * i for i in range(1, 8))


def test_glu_mm_refusals():
    def call(code=1, offsets=OFF, transpose_w=False, act="silu", **kw):
        a = dict(x=mat(A, 8, 16), w_gate=mat(B, 16, 24, groups=3), w_up=mat(C, 16, 24, groups=3), out=mat(D, 8, 24),
                 gate=mat(E, 8, 24), up=mat(F, 8, 24))
        a.update(kw)
        refused(code, L.ciera_glu_mm, a["x"], a["w_gate"], a["w_up"], a["out"], offsets=offsets,
                transpose_w=transpose_w, act=act, gate=a["gate"], up=a["up"])

    call(x=mat(A, 8, 17))                                       # contraction differs
    call(w_up=mat(C, 16, 25, groups=3))                         # the weights' shapes differ
    call(w_up=mat(C, 16, 24, groups=2))
    call(w_up=mat(C, 16, 24, F16, groups=3))
    call(out=mat(D, 8, 16))
    call(gate=mat(E, 7, 24))
    call(up=mat(F, 8, 24, F32))                                 # not out's type
    call(out=mat(D, 8, 24, F16), gate=mat(E, 8, 24, F16), up=mat(F, 8, 24, F16))
    call(transpose_w=True)
    call(act=3)
    call(act=0)
    call(gate=None)                                             # both or neither
    call(up=None)
    call(x=mat(A, 8, 16, groups=2))
    call(offsets=None)
    call(offsets=OFF + 2)
    for name in ("x", "w_gate", "w_up", "out", "gate", "up"):   # null, then misaligned
        rows, cols, groups = (16, 24, 3) if name.startswith("w_") else (8, 16 if name == "x" else 24, 1)
        call(**{name: mat(0, rows, cols, groups=groups)})
        call(**{name: mat(A + 1, rows, cols, groups=groups)})
    size = 8 * 24 * 2
    for at in (A + 8 * 16 * 2 - 2, B - size + 2, C + 100, E + 2, F - 2, OFF - size + 4):
        call(out=mat(at, 8, 24))                                # over an input, another output or the offsets
    call(gate=mat(F + 2, 8, 24))
    call(out=mat(D, 8, 24, ld=23))
    call(gate=mat(E, 8, 24, ld=23))
    call(w_gate=mat(B, 16, 24, groups=65537), w_up=mat(C, 16, 24, groups=65537), code=3)
    call(x=mat(A, 1 << 30, 16), out=mat(D, 1 << 30, 24), code=3)
    with pytest.raises(ValueError, match="act"):
        L.ciera_glu_mm(mat(A, 8, 16), mat(B, 16, 24), mat(C, 16, 24), mat(D, 8, 24), act="relu", stream=0)


def test_glu_grad_refusals():
    def call(code=1, offsets=OFF, transpose_w=False, act="gelu", **kw):
        a = dict(dy=mat(A, 8, 16), w_down=mat(B, 16, 24, groups=3), gate=mat(C, 8, 24), up=mat(D, 8, 24),
                 dgate=mat(E, 8, 24), dup=mat(F, 8, 24))
        a.update(kw)
        refused(code, L.ciera_glu_grad, a["dy"], a["w_down"], a["gate"], a["up"], a["dgate"], a["dup"],
                offsets=offsets, transpose_w=transpose_w, act=act)

    call(dy=mat(A, 8, 17))
    call(w_down=mat(B, 16, 25, groups=3))
    call(w_down=mat(B, 16, 24, F16, groups=3))
    call(transpose_w=True)
    call(act=7)
    call(offsets=None)
    call(offsets=OFF + 1)
    for name in ("gate", "up", "dgate", "dup"):
        call(**{name: mat(0, 8, 24)})
        call(**{name: mat(A + 1, 8, 24)})
        call(**{name: mat(0x9000000, 9, 24)})
        call(**{name: mat(0x9000000, 8, 24, F32)})              # the four are of one type
        call(**{name: mat(0x9000000, 8, 24, groups=2)})
    same = {n: mat(a, 8, 24, F16) for n, a in (("gate", C), ("up", D), ("dgate", E), ("dup", F))}
    call(**same)                                                # neither dy's type nor fp32
    for at in (A, B + 40, C, D + 2, F - 2, OFF - 8):
        call(dgate=mat(at, 8, 24))                              # in place of gate: not allowed either
    call(dup=mat(E + 2, 8, 24))
    call(dup=mat(F, 8, 24, ld=23))
    call(w_down=mat(B, 16, 24, groups=65537), code=3)


def test_glu_xgrad_refusals():
    def call(code=1, offsets=OFF, transpose_w=False, **kw):
        a = dict(dgate=mat(A, 8, 16), dup=mat(B, 8, 16), w_gate=mat(C, 16, 24, groups=3), w_up=mat(D, 16, 24, groups=3),
                 out=mat(E, 8, 24))
        a.update(kw)
        refused(code, L.ciera_glu_xgrad, a["dgate"], a["dup"], a["w_gate"], a["w_up"], a["out"], offsets=offsets,
                transpose_w=transpose_w)

    call(dup=mat(B, 8, 17))
    call(dup=mat(B, 8, 16, F16))
    call(dup=mat(B, 9, 16))
    call(dgate=mat(A, 8, 17), dup=mat(B, 8, 17))
    call(w_up=mat(D, 24, 16, groups=3))
    call(transpose_w=True)
    call(out=mat(E, 8, 16))
    call(out=mat(E, 8, 24, F16))
    call(offsets=None)
    call(offsets=OFF + 3)
    for at in (A, B + 8, C + 16, D - 2, OFF - 8, 0, E + 1):
        call(out=mat(at, 8, 24))
    call(w_gate=mat(C, 16, 24, groups=65537), w_up=mat(D, 16, 24, groups=65537), code=3)


def test_outputs_side_by_side():
    """Columns of one buffer pass the checks of overlap (no group: nothing is launched, but the
    sizes still are looked at) only where no element is shared."""
    lib = L._binding._lib

    def grad(gate, up, dgate, dup):
        return lib.ciera_glu_grad(*(ctypes.byref(m) for m in (mat(A, 8, 16), mat(B, 16, 24, groups=3))), 0, 1, OFF,
                                  *(ctypes.byref(m) for m in (gate, up, dgate, dup)), None)

    def cols(i, width=24, ld=96):
        return mat(0x9000000 + 2 * i, 8, width, ld=ld)

    # what shares elements is refused before any launch, so these are safe without a device
    assert grad(cols(0), cols(24), cols(48), cols(71)) == 1
    assert grad(cols(0), cols(24), cols(48), cols(73)) == 1      # wraps into the next row's gate
    assert grad(cols(0), cols(24), cols(24), cols(72)) == 1
    assert grad(cols(0), cols(24), cols(48), cols(72, ld=97)) == 1
    assert grad(cols(96), cols(24), cols(0), cols(1)) == 1


GQ = dict(codes=0x100000, scales=0x200000, zeros=0x300000)


def gq(groups=2, rows=40, cols=100, block=64, dtype=BF, reserved=0, **at):
    p = dict(GQ, **at)
    return L.Gq(p["codes"], p["scales"], p["zeros"], groups, block, dtype, reserved, rows, cols)


def test_gq_refusals():
    assert L.ciera_gq_sizes(2, 40, 100, 64) == (2 * 40 * 64, 2 * 40 * 2 * 2, 2 * 40 * 2)
    assert L.ciera_gq_sizes(1, 3, 129, 32) == (3 * 128, 3 * 8 * 2, 3 * 8)
    assert L.ciera_gq_sizes(0, 3, 5) == L.ciera_gq_sizes(3, 0, 5) == L.ciera_gq_sizes(3, 5, 0) == (0, 0, 0)
    for args in ((1 << 30, 1, 1), (1, 1 << 30, 1), (1, 1, 1 << 30), ((1 << 30) - 1, (1 << 30) - 1, 128)):
        with pytest.raises(L.CieraError) as e:
            L.ciera_gq_sizes(*args)
        assert e.value.code == 3
    for block in (0, 16, 48, 256):
        with pytest.raises(L.CieraError) as e:
            L.ciera_gq_sizes(1, 8, 8, block)
        assert e.value.code == 1
    x = mat(A, 40, 100, groups=2)
    bad = [gq(rows=41), gq(cols=99), gq(groups=1), gq(block=96), gq(dtype=F32), gq(reserved=1), gq(codes=0x100008),
           gq(codes=0), gq(scales=0), gq(scales=0x200002), gq(zeros=0x300002), gq(codes=A), gq(scales=A + 16),
           gq(zeros=A + 16), gq(scales=0x100000 + 5116), gq(zeros=0x200000 + 316), gq(zeros=0x100000)]
    for q in bad:
        refused(1, L.ciera_gq_quantize, x, q)
    refused(1, L.ciera_gq_quantize, x, gq(), axis=0)                # q is not the transpose
    refused(1, L.ciera_gq_quantize, mat(A, 100, 40, groups=2), gq(), axis=1)
    assert L._binding._lib.ciera_gq_quantize(ctypes.byref(x), 2, ctypes.byref(gq()), None) == 1
    with pytest.raises(ValueError, match="axis"):
        L.ciera_gq_quantize(x, gq(), axis=2)
    refused(1, L.ciera_gq_dequantize, gq(), mat(A, 40, 101, groups=2))
    for at in (0x100000, 0x200000 + 316, 0x300000 - 40 * 100 * 4 + 2, 0, A + 1):
        refused(1, L.ciera_gq_dequantize, gq(), mat(at, 40, 100, groups=2))


def test_gq_product_refusals():
    def mm(code=1, x=None, w=None, out=None, offsets=OFF):
        refused(code, L.ciera_gq_mm, x or mat(A, 8, 100), w or gq(), out or mat(B, 8, 40), offsets=offsets)

    def glu(code=1, w_up=None, act="silu", out=None, **kw):
        up = w_up or gq(codes=0x500000, scales=0x600000, zeros=0x700000)
        refused(code, L.ciera_gq_glu, mat(A, 8, 100), gq(**kw), up, out or mat(B, 8, 40), offsets=OFF, act=act)

    mm(x=mat(A, 8, 99))
    mm(x=mat(A, 8, 100, F32), out=mat(B, 8, 40, F32))
    mm(x=mat(A, 8, 100, groups=2))
    mm(out=mat(B, 8, 41))
    mm(out=mat(B, 7, 40))
    mm(out=mat(B, 8, 40, F16))
    mm(out=mat(B, 8, 40, ld=39))
    mm(offsets=None)
    mm(offsets=OFF + 2)
    mm(w=gq(block=31))
    mm(w=gq(codes=0))
    for at in (A, 0x100000, 0x200000, 0x300000, OFF - 8, 0, B + 1):
        mm(out=mat(at, 8, 40))
    mm(w=gq(groups=65537, codes=0x10000000, scales=0x90000000, zeros=0xa0000000), code=3)
    other = dict(codes=0x500000, scales=0x600000, zeros=0x700000)
    glu(w_up=gq(rows=41, **other))
    glu(w_up=gq(block=32, **other))
    glu(w_up=gq(dtype=F16, **other))
    glu(w_up=gq(groups=3, **other))
    glu(w_up=gq(codes=0x500000, scales=0x600000, zeros=None))      # both or neither
    glu(w_up=gq(codes=0x500004, scales=0x600000))
    glu(act=5)
    glu(out=mat(0x500000, 8, 40))
    glu(out=mat(0x700000, 8, 40))


def test_null_structures_are_invalid():
    lib = L._binding._lib
    m, q = ctypes.byref(mat(A, 8, 8)), ctypes.byref(gq(1, 8, 8))
    for i in range(4):
        t = [m] * 4
        t[i] = None
        assert lib.ciera_glu_mm(t[0], t[1], t[2], 0, 1, None, t[3], None, None, None) == 1
    for i in range(6):
        t = [m] * 6
        t[i] = None
        assert lib.ciera_glu_grad(t[0], t[1], 0, 1, None, t[2], t[3], t[4], t[5], None) == 1
    for i in range(5):
        t = [m] * 5
        t[i] = None
        assert lib.ciera_glu_xgrad(t[0], t[1], t[2], t[3], 0, None, t[4], None) == 1
    for x, w, u, o in ((None, q, q, m), (m, None, q, m), (m, q, None, m), (m, q, q, None)):
        assert lib.ciera_gq_glu(x, w, u, 1, None, o, None) == 1
        if u is not None:
            assert lib.ciera_gq_mm(x, w, None, o, None) == 1
    for x, w in ((None, q), (m, None)):
        assert lib.ciera_gq_quantize(x, 1, w, None) == 1
        assert lib.ciera_gq_dequantize(w, x, None) == 1
    assert lib.ciera_gq_sizes(1, 1, 1, 32, None, None, None) == 1


def test_nothing_to_write_needs_no_pointers():
    none = dict(stream=0)
    L.ciera_glu_mm(mat(0, 0, 16), mat(0, 16, 24, groups=3), mat(0, 16, 24, groups=3), mat(0, 0, 24), **none)
    L.ciera_glu_mm(mat(0, 8, 16), mat(0, 16, 0), mat(0, 16, 0), mat(0, 8, 0), gate=mat(0, 8, 0), up=mat(0, 8, 0), **none)
    L.ciera_glu_mm(mat(0, 8, 16), mat(0, 16, 24, groups=0), mat(0, 16, 24, groups=0), mat(0, 8, 24), **none)
    e = mat(0, 0, 24)
    L.ciera_glu_grad(mat(0, 0, 16), mat(0, 16, 24, groups=2), e, e, e, e, **none)
    L.ciera_glu_xgrad(mat(0, 0, 16), mat(0, 0, 16), mat(0, 16, 24), mat(0, 16, 24), e, **none)
    z = dict(codes=0, scales=0, zeros=0)
    L.ciera_gq_quantize(mat(0, 0, 16), gq(1, 0, 16, **z), **none)
    L.ciera_gq_dequantize(gq(0, 3, 16, **z), mat(0, 3, 16, groups=0), **none)
    L.ciera_gq_mm(mat(0, 0, 16), gq(2, 3, 16, **z), mat(0, 0, 3), **none)
    L.ciera_gq_glu(mat(0, 8, 16), gq(2, 0, 16, **z), gq(2, 0, 16, **z), mat(0, 8, 0), **none)


def test_binding_refuses_tensors_it_would_misread():
    need = L.ciera_gq_sizes(1, 8, 100, 32)
    with pytest.raises(ValueError, match="uint8"):
        L.gq_item(torch.zeros(need[0], dtype=torch.int8), 0x1000, None, 1, 8, 100, 32, BF)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        L.gq_item(0x1000, torch.zeros(need[1] // 2, dtype=torch.float32), None, 1, 8, 100, 32)
    with pytest.raises(ValueError, match="as scale_dtype says"):
        L.gq_item(0x1000, torch.zeros(need[1] // 2, dtype=torch.float16), None, 1, 8, 100, 32, BF)
    with pytest.raises(ValueError, match="scale_dtype"):
        L.gq_item(0x1000, 0x2000, None, 1, 8, 100, 32)
    with pytest.raises(ValueError, match="not on a GPU"):
        L.gq_item(torch.zeros(need[0], dtype=torch.uint8), 0x1000, None, 1, 8, 100, 32, BF)
    from lossless_weight_compression_amd.layer import GqMatrix
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        GqMatrix(8, 100, dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError, match="both, or nothing"):
        GqMatrix(8, 100, codes=torch.zeros(1))
    with pytest.raises(ValueError, match="both, or nothing"):
        GqMatrix(8, 100, zeros=torch.zeros(1))
    with pytest.raises(L.CieraError):
        GqMatrix(8, 100, block=100, device="cpu")


def test_binding_refuses_another_device(monkeypatch):
    class Elsewhere:
        dtype, shape, is_cuda, device = torch.bfloat16, (8, 16), True, torch.device("cuda", 1)
        stride = staticmethod(lambda *a: (16, 1)[a[0]] if a else (16, 1))
        numel = staticmethod(lambda: 128)
        data_ptr = staticmethod(lambda: A)
        get_device = staticmethod(lambda: 1)
        is_contiguous = staticmethod(lambda: True)

    class Quantised:
        codes, item = Elsewhere(), gq(1, 8, 16)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    m, w = mat(A, 8, 16), mat(B, 16, 24)
    for call in (lambda: L.ciera_gq_quantize(m, Quantised(), stream=0),
                 lambda: L.ciera_gq_dequantize(Quantised(), m, stream=0),
                 lambda: L.ciera_gq_mm(m, Quantised(), mat(C, 8, 8), stream=0),
                 lambda: L.ciera_gq_glu(m, gq(1, 8, 16), Quantised(), mat(C, 8, 8), stream=0),
                 lambda: L.ciera_glu_mm(m, w, w, mat(C, 8, 24), gate=Elsewhere(), up=mat(D, 8, 24), stream=0),
                 lambda: L.ciera_glu_grad(Elsewhere(), w, m, m, m, m, stream=0),
                 lambda: L.ciera_glu_xgrad(m, Elsewhere(), w, w, m, stream=0)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()


@pytest.mark.parametrize("stream", [None, 0x5000, "side"])
def test_results_are_allocated_on_the_stream_that_writes_them(stream, monkeypatch):
    from lossless_weight_compression_amd import layer
    active, made, real = [None], [], torch.empty

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            active.append(self.s)

        def __exit__(self, *a):
            active.pop()

    def empty(*a, **kw):
        made.append(active[-1])
        return real(*a, **{**kw, "device": "cpu"})

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, **kw: handle)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(layer.B, "gq_item", lambda *a: None)
    for name in ("ciera_gq_quantize", "ciera_gq_dequantize"):
        monkeypatch.setattr(layer.B, name, lambda *a: made.append(a[-1]))
    q = layer.GqMatrix(8, 128)
    made.clear()
    q.dequantize(stream=stream)
    assert made == [stream, stream]
    made.clear()
    codec = layer.LayerCodec.__new__(layer.LayerCodec)
    codec.device = "cpu"
    monkeypatch.setattr(layer.LayerCodec, "stack", lambda self, idx: torch.zeros(2, 128, 8))
    assert codec.quantize_groups([0, 1], stream=stream).rows == 8
    assert made == [stream] * 4                            # codes, scales, zeros, the call
    made.clear()
    codec.quantize_groups([0, 1], zeros=False, stream=stream)
    assert made == [stream] * 3
    made.clear()
    codec.quantize_groups([0, 1], into=q, stream=stream)
    assert made == [stream]
    with pytest.raises(ValueError, match="axis"):
        codec.quantize_groups([0, 1], axis=2)
