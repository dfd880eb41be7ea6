"""What the expert products and the 4-bit operators refuse, before any device
call (fake addresses, CPU tensors)."""
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


X, W, OUT, OFF = 0x1000000, 0x2000000, 0x3000000, 0x4000000


def test_group_mm_refusals():
    def call(x=None, w=None, out=None, offsets=OFF, transpose_w=False, code=1):
        refused(code, L.ciera_group_mm, x or mat(X, 8, 16), w or mat(W, 16, 24, groups=3), out or mat(OUT, 8, 24),
                offsets=offsets, transpose_w=transpose_w)

    call(x=mat(X, 8, 17))                                  # contraction differs
    call(out=mat(OUT, 9, 24))                              # rows differ
    call(out=mat(OUT, 8, 16))                              # columns differ
    call(transpose_w=True)                                 # w is [K, N], not [N, K]
    call(x=mat(X, 8, 16, F16))                             # types differ
    call(x=mat(X, 8, 16, F32), w=mat(W, 16, 24, F32, 3), out=mat(OUT, 8, 24, F32))
    call(out=mat(OUT, 8, 24, F16))                         # neither x's type nor fp32
    call(x=mat(X, 8, 16, 9))                               # no such type
    call(x=mat(X, 8, 16, groups=2))                        # x is one matrix
    call(out=mat(OUT, 8, 24, ld=23))                       # output rows overlap
    call(offsets=None)                                     # several groups need offsets
    call(offsets=OFF + 2)                                  # misaligned offsets
    call(x=mat(0, 8, 16))                                  # null operand
    call(out=mat(OUT + 1, 8, 24))                          # misaligned for its type
    call(out=mat(X + 2 * 8 * 16 - 2, 8, 24))               # starts in x's last element
    call(out=mat(W - 2 * 8 * 24 + 2, 8, 24))               # ends in w's first element
    call(x=mat(X, 1 << 30, 16), out=mat(OUT, 1 << 30, 24), code=3)
    call(x=mat(X, 8, 16, ld=1 << 62), code=3)
    call(w=mat(W, 16, 24, groups=65537), code=3)           # more groups than a product takes


def test_group_wgrad_refusals():
    def call(x=None, dy=None, out=None, offsets=OFF, code=1):
        refused(code, L.ciera_group_wgrad, x or mat(X, 8, 16), dy or mat(W, 8, 24), out or mat(OUT, 16, 24, groups=3),
                offsets=offsets)

    call(dy=mat(W, 9, 24))
    call(out=mat(OUT, 24, 16, groups=3))
    call(out=mat(OUT, 16, 24, groups=3, gs=16 * 24 - 1))   # output matrices overlap
    call(out=mat(OUT, 16, 24, groups=3, gs=0))
    call(out=mat(OUT, 16, 24, F16, groups=3))
    call(dy=mat(W, 8, 24, F16))
    call(dy=mat(W, 8, 24, groups=2))
    call(offsets=None)
    call(dy=mat(0, 8, 24))
    call(out=mat(X, 16, 24, groups=3))
    call(x=mat(X, 8, 1 << 30), out=mat(OUT, 1 << 30, 24, groups=3), code=3)
    call(out=mat(OUT, 16, 24, groups=65537), code=3)


def test_mx_refusals():
    q = L.Mx(0x100000, 0x200000, 2, 0, 40, 100)
    assert L.ciera_mx_sizes(2, 40, 100) == (2 * 40 * 64, 2 * 40 * 4)
    assert L.ciera_mx_sizes(1, 3, 129) == (3 * 128, 3 * 8)
    assert L.ciera_mx_sizes(0, 3, 5) == L.ciera_mx_sizes(3, 0, 5) == L.ciera_mx_sizes(3, 5, 0) == (0, 0)
    x = mat(X, 40, 100, groups=2)
    refused(1, L.ciera_mx_quantize, x, q, axis=0)                                   # q is not the transpose
    refused(1, L.ciera_mx_quantize, mat(X, 100, 40, groups=2), q, axis=1)
    refused(1, L.ciera_mx_quantize, mat(X, 40, 100), q)                             # groups differ
    refused(1, L.ciera_mx_quantize, x, L.Mx(0x100008, 0x200000, 2, 0, 40, 100))     # codes misaligned
    refused(1, L.ciera_mx_quantize, x, L.Mx(0x100000, 0x200002, 2, 0, 40, 100))     # scales misaligned
    refused(1, L.ciera_mx_quantize, x, L.Mx(0x100000, 0x100000 + 5116, 2, 0, 40, 100))  # scales in the codes
    refused(1, L.ciera_mx_quantize, x, L.Mx(X, 0x200000, 2, 0, 40, 100))            # codes over x
    refused(1, L.ciera_mx_quantize, x, L.Mx(0x100000, 0x200000, 2, 1, 40, 100))     # reserved
    refused(1, L.ciera_mx_quantize, x, L.Mx(0, 0x200000, 2, 0, 40, 100))
    refused(1, L.ciera_mx_dequantize, q, mat(OUT, 40, 101, groups=2))
    refused(1, L.ciera_mx_dequantize, q, mat(0x100000, 40, 100, groups=2))
    with pytest.raises(ValueError):
        L.ciera_mx_quantize(x, q, axis=2)
    assert L._binding._lib.ciera_mx_quantize(ctypes.byref(x), 2, ctypes.byref(q), None) == 1
    a, b = L.Mx(0x100000, 0x200000, 1, 0, 8, 100), L.Mx(0x300000, 0x400000, 3, 0, 24, 100)

    def mm(a=a, b=b, out=None, offsets=OFF, code=1):
        refused(code, L.ciera_mx_mm, a, b, out or mat(OUT, 8, 24), offsets=offsets)

    mm(a=L.Mx(0x100000, 0x200000, 1, 0, 8, 99))
    mm(a=L.Mx(0x100000, 0x200000, 2, 0, 8, 100))
    mm(out=mat(OUT, 8, 23))
    mm(out=mat(OUT, 7, 24))
    mm(out=mat(OUT, 8, 24, 7))
    mm(offsets=None)
    mm(offsets=OFF + 1)
    mm(out=mat(0x300000, 8, 24))
    mm(out=mat(0x200000 + 8 * 4 - 2, 8, 24))
    mm(a=L.Mx(0x100000, 0x200000, 1, 0, 1 << 30, 100), out=mat(OUT, 1 << 30, 24), code=3)
    mm(b=L.Mx(0x300000, 0x4000000, 65537, 0, 24, 100), code=3)
    for args in ((1 << 30, 1, 1), (1, 1 << 30, 1), (1, 1, 1 << 30), ((1 << 30) - 1, (1 << 30) - 1, 128)):
        with pytest.raises(L.CieraError) as e:
            L.ciera_mx_sizes(*args)
        assert e.value.code == 3
    assert L._binding._lib.ciera_mx_sizes(1, 1, 1, None, None) == 1


def test_null_structures_are_invalid():
    lib, m, q = L._binding._lib, mat(X, 8, 8), L.Mx(0x100000, 0x200000, 1, 0, 8, 8)
    m, q = ctypes.byref(m), ctypes.byref(q)
    for args in ((None, m), (m, None)):
        assert lib.ciera_mx_quantize(args[0], 1, q if args[1] else None, None) == 1
        assert lib.ciera_mx_dequantize(q if args[0] else None, args[1], None) == 1
    for i in range(3):
        t = [m, m, m]
        t[i] = None
        assert lib.ciera_group_mm(t[0], t[1], 0, None, t[2], None) == 1
        assert lib.ciera_group_wgrad(t[0], t[1], None, t[2], None) == 1
        u = [q, q, m]
        u[i] = None
        assert lib.ciera_mx_mm(u[0], u[1], None, u[2], None) == 1


def test_nothing_to_write_needs_no_pointers():
    L.ciera_group_mm(mat(0, 0, 16), mat(0, 16, 24, groups=3), mat(0, 0, 24), offsets=None, stream=0)
    L.ciera_group_mm(mat(0, 8, 16), mat(0, 16, 0, groups=3), mat(0, 8, 0), offsets=None, stream=0)
    L.ciera_group_mm(mat(0, 8, 16), mat(0, 16, 24, groups=0), mat(0, 8, 24), offsets=None, stream=0)
    L.ciera_group_wgrad(mat(0, 8, 0), mat(0, 8, 24), mat(0, 0, 24, groups=3), offsets=None, stream=0)
    L.ciera_group_wgrad(mat(0, 8, 16), mat(0, 8, 24), mat(0, 16, 24, groups=0), offsets=None, stream=0)
    L.ciera_mx_quantize(mat(0, 0, 16), L.Mx(0, 0, 1, 0, 0, 16), stream=0)
    L.ciera_mx_dequantize(L.Mx(0, 0, 0, 0, 3, 16), mat(0, 3, 16, groups=0), stream=0)
    L.ciera_mx_mm(L.Mx(0, 0, 1, 0, 0, 16), L.Mx(0, 0, 2, 0, 3, 16), mat(0, 0, 3), stream=0)


def test_binding_refuses_tensors_it_would_misread():
    a = torch.zeros(8, 16, dtype=torch.bfloat16)
    for t, msg in ((a, "not on a GPU"), (a.t(), "not adjacent"), (a.int(), "dtype"), (a[0], "dimensions"),
                   (a[None, None], "dimensions"), (a.double(), "dtype")):
        with pytest.raises(ValueError, match=msg):
            L.matrix_item(t, "x")
    with pytest.raises(ValueError, match="bytes"):
        L.mx_item(torch.zeros(8, 64), 0x1000, 1, 8, 100)
    with pytest.raises(ValueError, match="not on a GPU"):
        L.mx_item(torch.zeros(8, 64, dtype=torch.uint8), 0x1000, 1, 8, 100)
    m = mat(X, 8, 16)
    assert L.matrix_item(m) is m
    with pytest.raises(ValueError, match="dtype"):
        L.ciera_group_mm(m, mat(W, 16, 24), mat(OUT, 8, 24), offsets=torch.zeros(2, dtype=torch.int64), stream=0)


def test_binding_refuses_another_device(monkeypatch):
    """Operands that lie on a device other than the current one."""
    class Elsewhere:
        dtype, shape, is_cuda, device = torch.bfloat16, (8, 16), True, torch.device("cuda", 1)
        stride = staticmethod(lambda *a: (16, 1)[a[0]] if a else (16, 1))
        numel = staticmethod(lambda: 128)
        data_ptr = staticmethod(lambda: X)
        get_device = staticmethod(lambda: 1)
        is_contiguous = staticmethod(lambda: True)
        element_size = staticmethod(lambda: 1)

    class Quantised:
        codes, item = Elsewhere(), L.Mx(0x100000, 0x200000, 1, 0, 8, 16)

    class Offsets(Elsewhere):
        dtype = torch.int32
        numel = staticmethod(lambda: 2)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    m = mat(X, 8, 16)
    for call in (lambda: L.matrix_item(Elsewhere(), "x"),
                 lambda: L.ciera_mx_quantize(m, Quantised(), stream=0),
                 lambda: L.ciera_mx_dequantize(Quantised(), m, stream=0),
                 lambda: L.ciera_group_mm(m, mat(W, 16, 24), mat(OUT, 8, 24), offsets=Offsets(), stream=0)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert L.matrix_item(Elsewhere(), "x").rows == 8


@pytest.mark.parametrize("at", ["first", "last", "within", "around"])
def test_outputs_over_the_offsets_are_refused(at):
    """The kernels read the offsets, of groups + 1 words, while they write the output."""
    def place(out_bytes, offset_bytes):
        return {"first": OUT - offset_bytes + 4,       # the last offset in the output's first bytes
                "last": OUT + out_bytes - 4,           # the first offset in its last bytes
                "within": OUT + 8,
                "around": OUT - 8}[at]

    groups = 3 if at != "around" else 400
    x, out = mat(X, 8, 16), mat(OUT, 8, 24)
    refused(1, L.ciera_group_mm, x, mat(W, 16, 24, groups=groups), out, offsets=place(8 * 24 * 2, 4 * groups + 4))
    refused(1, L.ciera_group_mm, x, mat(W, 24, 16, groups=groups), out, offsets=place(8 * 24 * 2, 4 * groups + 4),
            transpose_w=True)
    refused(1, L.ciera_mx_mm, L.Mx(0x100000, 0x200000, 1, 0, 8, 100), L.Mx(0x300000, 0x400000, groups, 0, 24, 100), out,
            offsets=place(8 * 24 * 2, 4 * groups + 4))
    groups = 3
    size = 3 * 16 * 24 * 2
    where = place(size, 16) if at != "around" else OUT + size // 2
    refused(1, L.ciera_group_wgrad, x, mat(W, 8, 24), mat(OUT, 16, 24, groups=3), offsets=where)


@pytest.mark.parametrize("stream", [None, 0x5000, "side"])
def test_results_are_allocated_on_the_stream_that_writes_them(stream, monkeypatch):
    """Memory that another stream has freed may still be in use there: what a call on
    `stream` makes and writes has to come from that stream's memory."""
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
    monkeypatch.setattr(layer.B, "mx_item", lambda *a: None)
    for name in ("ciera_mx_quantize", "ciera_mx_dequantize"):
        monkeypatch.setattr(layer.B, name, lambda *a: made.append(a[-1]))
    q = layer.MxMatrix(8, 128)
    made.clear()
    q.dequantize(stream=stream)
    assert made == [stream, stream]
    made.clear()
    codec = layer.LayerCodec.__new__(layer.LayerCodec)
    codec.device = "cpu"
    monkeypatch.setattr(layer.LayerCodec, "stack", lambda self, idx: torch.zeros(2, 128, 8))
    assert codec.quantize([0, 1], stream=stream).rows == 8
    assert made == [stream] * 3                            # codes, scales, the call
    made.clear()
    codec.quantize([0, 1], into=q, stream=stream)
    assert made == [stream]
