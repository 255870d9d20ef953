"""How the linear layers and the norms at the residual stream are called: other streams and devices, captured graphs side by
side, tensors of more than 2^31 elements."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp8_ref as ref
import quantized_sparse_moe_router_gb300 as fw
from quantized_sparse_moe_router_gb300 import attention

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def rand(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def layer(T, K, N):
    return rand(T, K).bfloat16(), *fw.quantize_fp8_weight(rand(N, K, seed=1))


def linear():
    T, K, N = 2000, 1024, 1536
    a = layer(T, K, N)
    return lambda **kw: fw.linear_fp8(*a, **kw), [T * N * 2, T * K + 8 * T * 4]


def quantize():
    x = rand(3000, 2048).bfloat16()
    return lambda **kw: fw.quantize_fp8(x, **kw)[0], [3000 * 2048, 3000 * 16 * 4]


def weight():
    w = rand(2048, 2048)
    return lambda **kw: fw.quantize_fp8_weight(w, **kw)[0], [2048 * 2048, 16 * 16 * 4]


def norm():
    y = rand(3000, 1024).bfloat16()
    n = torch.ones(1024, device=DEV)
    return lambda **kw: fw.norm_residual(y, norm=n, **kw)[1], [3000 * 1024 * 2]


def norm_codes():
    y = rand(3000, 1024).bfloat16()
    return lambda **kw: fw.norm_residual(y, y, fp8=True, **kw)[1][0], [3000 * 1024 * 2, 3000 * 1024, 3000 * 8 * 4]


@pytest.mark.parametrize("made", [linear, quantize, weight, norm, norm_codes])
def test_memory_of_another_streams_call_is_not_the_current_streams(made):
    call, sizes = made()
    side = torch.cuda.Stream()
    want = call().clone()
    call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 3, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    copies = [torch.zeros_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # some 0.2 s, then the held memory is read, and is free for what the current stream does next
    for t, to in zip(held, copies):
        to.copy_(t)
    del held, t, to
    got = call(stream=side.cuda_stream)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # (it was still asleep: the test shows something)
    torch.cuda.synchronize()
    assert all((x == 3).all() for x in copies)
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_calls_refuse_tensors_of_another_device(monkeypatch):
    """Each call asks, before it makes or launches anything."""
    calls = [made()[0] for made in (linear, quantize, weight, norm, norm_codes)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(attention, "_several", True)
    for call in calls:
        call()
    monkeypatch.setattr(attention, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="cuda:0, the current device is cuda:1"):
            call()


@pytest.mark.parametrize("T", [1, 16, 60, 300])
def test_two_graphs_at_once(T):
    """Two captured chains of norm, linear layer and norm, replayed on two streams at once, again and again: each has its own workspace."""
    K, N = 1152, 640
    n = 1 + 0.1 * rand(K)

    def chain(seed):
        x, w = rand(T, K, seed=seed).bfloat16(), fw.quantize_fp8_weight(rand(N, K, seed=seed + 1))
        back = fw.quantize_fp8_weight(rand(K, N, seed=seed + 2))

        def step():
            r, (codes, scales) = fw.norm_residual(x, x, norm=n, fp8=True)
            y = fw.linear_fp8(fw.linear_fp8(codes, *w, x_scale=scales), *back)
            return fw.norm_residual(y, r, norm=n, post_norm=n)

        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        return x, w, back, g, got, want

    chains = [chain(5), chain(50)]
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(20):
        for (_, _, _, g, got, _), s in zip(chains, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, _, _, got, want in chains:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 16, 40, 64, 200])
def test_behind_the_experts(T):
    """Linear layers that follow a step of the fused experts at once, and the other way round: each has the tensor memory it needs."""
    H, I, E, k = 512, 128, 16, 2
    q8 = lambda r, c, s: torch.stack([fw.quantize_q8_0(rand(r, c, seed=s + e) * c ** -0.5) for e in range(E)])  # noqa: E731
    moe = fw.MoELayer(H, I, E, k, T_max=16, weights=dict(router_w=rand(E, H) * H ** -0.5, w_gate=q8(I, H, 10), w_up=q8(I, H, 40), w_down=q8(H, I, 70)))
    x16 = rand(16, H, seed=3).bfloat16()
    x, w, ws = layer(T, H, 1024)
    codes, scales = fw.quantize_fp8(x)
    want, want_moe = fw.linear_fp8(codes, w, ws, x_scale=scales), moe.forward(x16)[1].clone()
    got = [(moe.forward(x16)[1].clone() if i % 10 == 9 else moe.forward(x16)[1], fw.linear_fp8(codes, w, ws, x_scale=scales)) for i in range(100)]
    torch.cuda.synchronize()
    moe.status()
    assert all(torch.equal(b, want) for _, b in got) and torch.equal(got[99][0], want_moe)
    moe.close()


def check_products(x, w, rows, cols, out, codes, scales):
    """The products of some tokens and some outputs (whole blocks of them)."""
    want, tol = ref.linear(bits(codes[rows]), f64(scales[:, rows]).T, bits(w[0][cols]), f64(w[1][cols.start // 128:(cols.stop + 127) // 128]))
    got = f64(out[rows][:, cols])
    assert (np.abs(got - want) <= tol + ref.BF16 * (np.abs(want) + tol)).all()


def test_more_than_2_31_outputs():
    T, K, N = 16500, 128, 131072 + 256
    x, w = rand(T, K).bfloat16(), fw.quantize_fp8_weight(rand(N, K, seed=1))
    out = fw.linear_fp8(x, *w)
    codes, scales = fw.quantize_fp8(x)
    for r in (0, T - 1):
        for c in (slice(0, 128), slice(N - 128, N)):
            check_products(x, w, slice(r, r + 1), c, out, codes, scales)


def test_more_than_2_31_weights():
    K, N = 16384, 131072 + 384
    w16 = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, N, 16384):
        w16[i:i + 16384] = rand(min(16384, N - i), K, seed=i).bfloat16()
    w = fw.quantize_fp8_weight(w16)
    c, s = ref.quantise(f64(w16[-128:]), 128)
    assert np.array_equal(bits(w[0][-128:]), c) and np.array_equal(w[1][-1:].cpu().numpy(), s)
    del w16
    for T in (3, 40, 130):
        x = rand(T, K).bfloat16()
        out = fw.linear_fp8(x, *w)
        codes, scales = fw.quantize_fp8(x)
        check_products(x, w, slice(0, T), slice(N - 128, N), out, codes, scales)
        check_products(x, w, slice(0, T), slice(0, 128), out, codes, scales)


def test_more_than_2_31_activations():
    T, H = 140000, 16384
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 20000):
        y[i:i + 20000] = rand(20000, H, seed=i).bfloat16()
    codes, scales = fw.quantize_fp8(y)
    some = [0, 65537, 131072, T - 1]
    c, s = ref.quantise(f64(y[some]), 1)
    assert np.array_equal(bits(codes[some]), c) and np.array_equal(scales[:, some].cpu().numpy().T, s)
    w = fw.quantize_fp8_weight(rand(64, H, seed=1))
    out = fw.linear_fp8(codes, *w, x_scale=scales)
    for r in some:
        check_products(y, w, slice(r, r + 1), slice(0, 64), out, codes, scales)
    del codes, scales, out
    norm = 1 + 0.1 * rand(H)
    small = fw.norm_residual(y[some], y[some], norm=norm, fp8=True)
    r, (codes, scales) = fw.norm_residual(y, y, norm=norm, fp8=True)
    assert torch.equal(r[some], small[0]) and torch.equal(codes[some].view(torch.uint8), small[1][0].view(torch.uint8))
    assert torch.equal(scales[:, some], small[1][1])
    del codes, scales
    r, h = fw.norm_residual(y, y, norm=norm)
    want = fw.norm_residual(y[some], y[some], norm=norm)
    assert torch.equal(r[some], want[0]) and torch.equal(h[some], want[1])
