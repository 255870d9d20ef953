"""How the calls of the 8-bit linear layers make their outputs: by torch's quicker way or, where it is missing or takes
other arguments, by torch.empty, with the same tensors."""
import pytest

torch = pytest.importorskip("torch")

import quantized_sparse_moe_router_gb300 as fw
from quantized_sparse_moe_router_gb300 import linear

MADE = [(0, 16, torch.bfloat16), (1, 1, torch.float32), (3, 4096, torch.float8_e4m3fn), (1, 777, torch.uint8)]


class Like:
    device = torch.device("cpu")


def of_other_arguments(size):
    raise AssertionError("not reached")


@pytest.mark.parametrize("way", [None, of_other_arguments])
def test_without_the_quicker_way(monkeypatch, way):
    monkeypatch.setattr(linear, "_empty_strided", way)
    for rows, cols, kind in MADE:
        t = linear._new(rows, cols, kind, Like, None)
        assert t.shape == (rows, cols) and t.dtype is kind and t.is_contiguous()
    assert linear._empty_strided is None


@pytest.mark.gpu
def test_both_ways_are_the_same(monkeypatch):
    like = torch.empty(1, device="cuda")
    quick = [linear._new(*m, like, None) for m in MADE]
    x = torch.randn(40, 256, device="cuda").bfloat16()
    w = fw.quantize_fp8_weight(torch.randn(64, 256, device="cuda"))
    with_quick = [fw.linear_fp8(x, *w), *fw.norm_residual(x, x)]
    monkeypatch.setattr(linear, "_empty_strided", of_other_arguments)
    plain = [linear._new(*m, like, None) for m in MADE]
    assert linear._empty_strided is None
    for a, b in zip(quick, plain):
        assert a.shape == b.shape and a.stride() == b.stride() and a.dtype is b.dtype and a.device == b.device
        assert a.requires_grad == b.requires_grad and type(a) is type(b) and a.untyped_storage().nbytes() == b.untyped_storage().nbytes()
    assert all(torch.equal(a, b) for a, b in zip(with_quick, [fw.linear_fp8(x, *w), *fw.norm_residual(x, x)]))
