"""Outputs whose rows lie apart at multiples of 16 bytes and end inside one: what follows a row's last output stays."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_sparse_moe_router_gb300 as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)

# few tokens; pairs of SMs 128 wide, sharing a tile, and 256 wide (each with N up to 7 below)
SIZES = [(1, 256, 384), (16, 2048, 136), (40, 256, 384), (100, 7168, 256), (70, 128, 8), (300, 512, 384), (500, 7168, 1536), (2048, 256, 2304), (4097, 128, 264)]


@pytest.mark.parametrize("T, K, N", SIZES)
@pytest.mark.parametrize("less", range(8))
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_what_follows_a_row_stays(T, K, N, less, kind):
    n = N - less
    g = torch.Generator(device=DEV).manual_seed(T + n)
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    w, ws = fw.quantize_fp8_weight(torch.randn(n, K, generator=g, device=DEV))
    want = fw.linear_fp8(x, w, ws, out_dtype=kind)
    wide = torch.full((T, N + 24), 7.0, dtype=kind, device=DEV)
    fw.linear_fp8(x, w, ws, out=wide[:, 8:8 + n])
    assert torch.equal(wide[:, 8:8 + n], want)
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + n:] == 7).all()
