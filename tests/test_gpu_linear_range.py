"""Linear layers in 8 bits whose two scales have a product that fp32 does not hold, or holds in fewer bits, while the
results are ordinary numbers: every kernel and every way of cutting the products up."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp8_ref as ref
import quantized_sparse_moe_router_gb300 as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)

# bf16 quantised in the kernel, codes of up to 16, 32, 64 and 128 tokens; pairs of SMs 128 wide, sharing a
# tile, and 256 wide; the last of few tokens with more than 32 blocks in a part of K
SHAPES = [(1, 1024, 384), (16, 2048, 300), (24, 1024, 384), (50, 1024, 256), (100, 512, 384), (300, 1024, 384), (300, 7168, 576), (2100, 384, 2304),
          (100, 7168, 256), (500, 7168, 1536), (2048, 4224, 2304), (40, 4224, 20000)]


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def normals(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device=DEV), lambda lo, hi, n: torch.exp2(torch.randint(lo, hi, (n,), generator=g, device=DEV).float())


def check(x, w, ws):
    codes, scales = fw.quantize_fp8(x)
    out = fw.linear_fp8(codes, w, ws, x_scale=scales, out_dtype=torch.float32)
    assert torch.equal(fw.linear_fp8(x, w, ws, out_dtype=torch.float32), out)
    want, tol = ref.linear(bits(codes), f64(scales).T, bits(w), f64(ws))
    got = f64(out)
    # (sums next to nothing: each addition of a block's is then off by half of fp32's smallest number)
    tol = tol + ref.FP32 * np.abs(want) + (x.shape[1] // 128 + 2) * 2.0 ** -150
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("T, K, N", SHAPES)
def test_products_of_small_scales(T, K, N):
    """Scale products from 2^-165 to 2^-110, block by block, against outputs of about 2^-110."""
    n, by = normals(T + N)
    nb = lambda v, m: v.repeat_interleave(128)[:m]  # noqa: E731
    x = (n(T, K) * nb(by(-70, -44, K // 128), K) * by(-6, 1, T)[:, None]).bfloat16()
    w, ws = fw.quantize_fp8_weight(n(N, K) * nb(by(-70, -44, K // 128), K) * nb(by(-6, 1, N // 128 + 1), N)[:, None])
    check(x, w, ws)


@pytest.mark.parametrize("T, K, N", SHAPES)
@pytest.mark.parametrize("a, b", [(110, -110), (-100, 100), (56, 60), (-20, 80), (-95, 20), (4, -90), (-62, -62), (-63, -63), (-66, -60), (-58, -68)])
def test_products_of_scales_far_from_one(T, K, N, a, b):
    n, _ = normals(T + N)
    x = (n(T, K) * 2.0 ** a).bfloat16()
    w, ws = fw.quantize_fp8_weight(n(N, K) * 2.0 ** b)
    check(x, w, ws)


@pytest.mark.parametrize("T, K, N", SHAPES)
@pytest.mark.parametrize("a, b", [(74, 74), (100, 46), (24, 122)])
def test_sums_of_nothing_under_large_scales(T, K, N, a, b):
    """Every product has a factor of zero, and the product of the scales is infinite."""
    n, _ = normals(T + N)
    even = (torch.arange(K, device=DEV) % 2 == 0).float()
    x = (n(T, K) * even * 2.0 ** a).bfloat16()
    w, ws = fw.quantize_fp8_weight(n(N, K) * (1 - even) * 2.0 ** b)
    assert torch.isinf(ws.max() * fw.quantize_fp8(x)[1].max())
    for kind in (torch.float32, torch.bfloat16):
        assert (fw.linear_fp8(x, w, ws, out_dtype=kind) == 0).all()


@pytest.mark.parametrize("T", [1, 24, 300])
def test_blocks_of_zeros(T):
    """Weights whose blocks are zeros, or have a scale of zero, beside others; an infinite activation still reaches its outputs."""
    K, N = 512, 384
    n, _ = normals(T)
    x, full = n(T, K).bfloat16(), n(N, K)
    full[128:256] = 0
    full[:, 128:256] = 0
    w, ws = fw.quantize_fp8_weight(full)
    check(x, w, ws)
    ws[1] = 0
    check(x, w, ws)
    x[0, 3] = float("inf")
    out = fw.linear_fp8(x, w, ws, out_dtype=torch.float32)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1:]).all()
