"""8-bit results of the norms, bit by bit, and the residual stream in fp32 on all of many rows."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp8_ref as ref
import quantized_sparse_moe_router_gb300 as fw

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("T", [1, 3, 44, 104])
def test_codes_of_the_examples_layer(T):
    """The layer's first norm to 8 bits is that of its bf16 result, quantised."""
    layer = ex.EightBitLayer()
    x = torch.randn(T, 512, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).bfloat16()
    codes, scales = fw.norm_residual(x, norm=layer.norm1, fp8=True)[1]
    want_c, want_s = fw.quantize_fp8(fw.norm_residual(x, norm=layer.norm1)[1])
    assert torch.equal(codes.view(torch.uint8), want_c.view(torch.uint8)) and torch.equal(scales, want_s)


@pytest.mark.parametrize("T, H", [(1000, 1032), (700, 2048), (4097, 2560), (999, 7168), (305, 32768)])
@pytest.mark.parametrize("post", [False, True])
def test_many_rows_of_an_fp32_residual(T, H, post):
    """r of every row: the sum's rounding, and in the norm before it H / 2 roundings of the sum of squares and eight more."""
    g = torch.Generator(device=DEV).manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    y, residual, weight = n(T, H).bfloat16(), 3 * n(T, H), 1 + 0.1 * n(H)
    gate = torch.sigmoid(n(T, 1))
    r, _ = fw.norm_residual(y, residual, norm=weight, post_norm=weight if post else None, gate=gate, scale=0.5)
    add = y.double()
    if post:
        add = add / (add.square().mean(1, keepdim=True) + 1e-6).sqrt() * weight.double()
    add = add * gate.double() * 0.5
    want = residual.double() + add
    off = (H / 2 + 8 if post else 3) * ref.FP32 * add.abs() + ref.FP32 * want.abs()
    assert r.dtype is torch.float32 and ((r.double() - want).abs() <= off * 1.001).all()
