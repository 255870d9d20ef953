"""Linear layers in 8 bits: blocks bit by bit, products against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp8_ref as ref
import quantized_sparse_moe_router_gb300 as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def tokens(T, K, seed, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return (n(T, K) * torch.exp(spread * n(K)) * torch.exp(spread * n(T, 1))).bfloat16()


def weights(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return n(N, K) * K ** -0.5 * torch.exp(n(N, 1))


def check(out, x, w, w_scale, x_scale=None, rows=None):
    """out against the definition, on all rows or those given."""
    if x_scale is None:
        xc, xs = ref.quantise(f64(x), 1)
    else:
        xc, xs = bits(x), x_scale.cpu().numpy().T
    rows = slice(None) if rows is None else rows
    want, tol = ref.linear(xc[rows], xs[rows], bits(w), w_scale.cpu().numpy())
    got = f64(out)[rows]
    tol = tol + (ref.BF16 if out.dtype is torch.bfloat16 else ref.FP32) * np.abs(want) * 1.001
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("T, K", [(1, 16), (1, 128), (3, 144), (17, 2048), (5, 4000), (1000, 400)])
def test_blocks_of_tokens(T, K):
    x = tokens(T, K, T + K, 2.0)
    x[0, :16] = 0
    codes, scales = fw.quantize_fp8(x)
    want_c, want_s = ref.quantise(f64(x), 1)
    assert np.array_equal(bits(codes), want_c)
    assert np.array_equal(scales.cpu().numpy().T, want_s)


def test_blocks_of_special_values():
    """Zeros, subnormals, the largest, infinities and NaN; a block of its own each."""
    x = torch.zeros(8, 256, dtype=torch.bfloat16, device=DEV)
    x[1, :3] = torch.tensor([1e-39, -2e-39, 5e-40])
    x[2, 5] = 2.0 ** -96
    x[3, :2] = torch.tensor([3.38e38, -1e38])
    x[4, 7] = float("inf")
    x[5, 130] = float("nan")
    x[6] = 1.0
    x[7, ::2] = -0.0
    codes, scales = fw.quantize_fp8(x)
    c, s = ref.quantise(f64(x), 1)
    got = scales.cpu().numpy().T
    assert np.array_equal(np.isnan(got), np.isnan(s)) and np.array_equal(got[~np.isnan(s)], s[~np.isnan(s)])
    fine = [0, 1, 2, 3, 6, 7]
    assert np.array_equal(bits(codes)[fine], c[fine])
    w, ws = fw.quantize_fp8_weight(weights(40, 256, 1))
    out = f64(fw.linear_fp8(x, w, ws, out_dtype=torch.float32))
    assert np.isnan(out[4]).all() and np.isnan(out[5]).all() and np.isfinite(out[fine]).all()
    assert (out[[0, 7]] == 0).all()


@pytest.mark.parametrize("N, K", [(1, 16), (128, 128), (130, 272), (1000, 2048)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_blocks_of_weights(N, K, kind):
    w = weights(N, K, N + K).to(kind)
    codes, scales = fw.quantize_fp8_weight(w)
    want_c, want_s = ref.quantise(f64(w), 128)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(bits(codes), want_c)


SHAPES = [(1, 16, 1), (1, 128, 128), (1, 2048, 5120), (2, 4000, 129), (7, 1040, 640), (8, 2048, 256), (9, 2048, 256), (16, 7168, 384), (17, 512, 1000),
          (31, 2064, 255), (33, 144, 127), (64, 2048, 2048), (65, 1152, 130), (100, 7168, 256), (128, 256, 4096), (129, 640, 300), (257, 4096, 512),
          (333, 4000, 2051), (512, 1024, 1024), (1000, 528, 777), (70, 7168, 128), (256, 16, 512), (257, 16, 513), (300, 2000, 5000), (2100, 384, 2304),
          (1300, 640, 4097), (4000, 272, 136)]


@pytest.mark.parametrize("T, K, N", SHAPES)
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_products(T, K, N, kind):
    x, (w, ws) = tokens(T, K, 1), fw.quantize_fp8_weight(weights(N, K, 2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fw.linear_fp8(x, w, ws, out_dtype=kind, status=status)
    check(out, x, w, ws)
    codes, scales = fw.quantize_fp8(x)
    same = fw.linear_fp8(codes, w, ws, x_scale=scales, out_dtype=kind, status=status)
    assert torch.equal(out, same)
    assert status.item() == 0


@pytest.mark.parametrize("T, K, N", [(300, 7168, 576), (300, 7168, 577), (130, 7168, 1024), (500, 7168, 1536), (257, 7168, 2047), (200, 7088, 1500), (513, 16400, 200)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_products_of_shared_tiles(T, K, N, kind):
    """Few tiles and a long K, which pairs of SMs then share; rows apart, and of no alignment."""
    x, (w, ws) = tokens(T, K, 1), fw.quantize_fp8_weight(weights(N, K, 2))
    out = fw.linear_fp8(x, w, ws, out_dtype=kind)
    check(out, x, w, ws)
    big = torch.full((T, N + 37), 7.0, dtype=kind, device=DEV)
    assert torch.equal(fw.linear_fp8(x, w, ws, out=big[:, 5:5 + N]), out)
    assert (big[:, :5] == 7).all() and (big[:, 5 + N:] == 7).all()


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_scales_far_apart(T):
    """Blocks whose scales differ by many powers of two, along K and over tokens and outputs."""
    K, N = 1024, 384
    g = torch.Generator(device=DEV).manual_seed(9)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    by = lambda c: torch.exp2(torch.randint(-20, 20, (c,), generator=g, device=DEV).float())  # noqa: E731
    x = (n(T, K) * by(K // 128).repeat_interleave(128) * by(T)[:, None]).bfloat16()
    w, ws = fw.quantize_fp8_weight(n(N, K) * by(K // 128).repeat_interleave(128) * by(N // 128).repeat_interleave(128)[:, None])
    check(fw.linear_fp8(x, w, ws, out_dtype=torch.float32), x, w, ws)


@pytest.mark.parametrize("T", [1, 16, 50, 200])
def test_views(T):
    """Rows apart in memory on both sides; what lies between output rows stays."""
    K, N = 640, 300
    wide = tokens(T, K + 72, 3)
    x = wide[:, 8:8 + K]
    w, ws = fw.quantize_fp8_weight(weights(N, K, 4))
    big = torch.full((T, N + 37), 7.0, dtype=torch.bfloat16, device=DEV)
    out = fw.linear_fp8(x, w, ws, out=big[:, 3:3 + N])
    check(out, x, w, ws)
    assert (big[:, :3] == 7).all() and (big[:, 3 + N:] == 7).all()
    codes, scales = fw.quantize_fp8(x)
    pitch = torch.zeros(T, K + 16, dtype=torch.uint8, device=DEV)
    pitch[:, :K] = codes.view(torch.uint8)
    assert torch.equal(fw.linear_fp8(pitch[:, :K].view(torch.float8_e4m3fn), w, ws, x_scale=scales), out)


@pytest.mark.parametrize("T", [1, 16, 64, 300])
def test_same_bits_each_time(T):
    x, (w, ws) = tokens(T, 4096, 5), fw.quantize_fp8_weight(weights(512, 4096, 6))
    first = fw.linear_fp8(x, w, ws, out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(fw.linear_fp8(x, w, ws, out_dtype=torch.float32), first)


def test_empty_and_streams():
    w, ws = fw.quantize_fp8_weight(weights(64, 256, 7))
    assert fw.linear_fp8(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV), w, ws).shape == (0, 64)
    assert fw.quantize_fp8(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV))[1].shape == (2, 0)
    side = torch.cuda.Stream()
    for T in (3, 100):
        x = tokens(T, 256, 8)
        want = fw.linear_fp8(x, w, ws)
        torch.cuda.synchronize()
        got = fw.linear_fp8(x, w, ws, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(got, want)


def test_captured():
    """Two layers in one graph, replayed on new inputs."""
    (w1, s1), (w2, s2) = fw.quantize_fp8_weight(weights(512, 256, 1)), fw.quantize_fp8_weight(weights(128, 512, 2))
    for T in (1, 90, 700):
        x, fresh = tokens(T, 256, 1), tokens(T, 256, 2)
        two = lambda v: fw.linear_fp8(fw.linear_fp8(v, w1, s1), w2, s2)  # noqa: E731
        two(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = two(x)
        x.copy_(fresh)
        graph.replay()
        assert torch.equal(y, two(fresh))
