"""LayerCodec.quantize_groups into memory that is there: its format is not silently another one than
asked for (CPU tensors, no device call)."""
import pytest
import torch

layer = pytest.importorskip("lossless_weight_compression_amd.layer")


@pytest.fixture
def codec(monkeypatch):
    """A codec whose stack is two matrices [128, 8]; what is quantised is noted down."""
    c = layer.LayerCodec.__new__(layer.LayerCodec)
    c.device, c.done = "cpu", []
    monkeypatch.setattr(layer.LayerCodec, "stack", lambda self, idx: torch.zeros(2, 128, 8))
    monkeypatch.setattr(layer.B, "gq_item", lambda *a: None)
    monkeypatch.setattr(layer.B, "ciera_gq_quantize", lambda x, q, axis, stream: c.done.append((q, axis, stream)))
    return c


def into(block=64, dtype=torch.float16, zeros=False):
    return layer.GqMatrix(8, 128, groups=2, block=block, dtype=dtype, with_zeros=zeros, device="cpu")


@pytest.mark.parametrize("asked,word", [(dict(block=32), "block"), (dict(block=128), "block"),
                                        (dict(scale_dtype=torch.bfloat16), "scale_dtype"), (dict(zeros=True), "zeros"),
                                        (dict(block=64, zeros=True), "zeros")])
def test_another_format_than_that_of_into_is_refused(codec, asked, word):
    with pytest.raises(ValueError, match=word):
        codec.quantize_groups([0, 1], into=into(), stream=0, **asked)
    assert codec.done == []


def test_zeros_that_into_has_are_not_dropped(codec):
    with pytest.raises(ValueError, match="zeros"):
        codec.quantize_groups([0, 1], into=into(zeros=True), zeros=False, stream=0)


@pytest.mark.parametrize("asked", [{}, dict(block=64), dict(scale_dtype=torch.float16), dict(zeros=False),
                                   dict(block=64, scale_dtype=torch.float16, zeros=False)])
def test_the_format_of_into(codec, asked):
    q = into()
    assert codec.quantize_groups([0, 1], into=q, stream=0, **asked) is q
    assert codec.done == [(q, 0, 0)]


def test_formats_of_new_copies(codec, monkeypatch):
    monkeypatch.setattr(layer, "_memory_of", lambda stream: torch.no_grad())
    q = codec.quantize_groups([0, 1], stream=0)
    assert (q.block, q.scales.dtype, q.zeros is not None) == (128, torch.bfloat16, True)
    q = codec.quantize_groups([0, 1], block=32, scale_dtype=torch.float16, zeros=False, stream=0)
    assert (q.block, q.scales.dtype, q.zeros is not None) == (32, torch.float16, False)
    with pytest.raises(ValueError, match="axis"):
        codec.quantize_groups([0, 1], axis=2)
