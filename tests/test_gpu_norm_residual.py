"""The norms at the residual stream with gate, scale and sum, against 64 bits."""
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
    return None if t is None else t.double().cpu().numpy()


def inputs(T, H, residual, gate, post, norm, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(y=n(T, H).bfloat16(), residual=None if residual is None else (3 * n(T, H)).to(residual),
                gate={"none": lambda: None, "channel": lambda: n(H), "channel16": lambda: n(1, H).bfloat16(), "token": lambda: n(T, 1).bfloat16(),
                      "token32": lambda: n(T, 1), "full": lambda: n(T, H).bfloat16(), "full32": lambda: n(T, H)}[gate](),
                post_norm=1 + 0.1 * n(H) if post else None, norm=1 + 0.1 * n(H) if norm else None)


def check(a, r, h, scale=1.0, eps=1e-6):
    want_r, want_h, big = ref.norm_residual(f64(a["y"]), f64(a["residual"]), f64(a["norm"]), f64(a["post_norm"]), f64(a["gate"]), scale, eps)
    H = a["y"].shape[1]
    # the row's sum of squares: H / (a thread's share) additions in any order, at most H of 2^-24, and half of that after the
    # root; the root itself, and the products with scale, gate and weight: 2^-22
    fp = (H / 2 + 8) * ref.FP32
    u = ref.FP32 if r.dtype is torch.float32 else ref.BF16
    assert (np.abs(f64(r) - want_r) <= u * np.abs(want_r) * 1.001 + fp * big).all()
    rel = fp * (1 if a["norm"] is None else 2)
    grow = 1.0 if a["norm"] is None else np.abs(f64(a["norm"])) / np.sqrt((want_r ** 2).mean(1, keepdims=True) + eps)
    if h is not None:
        assert (np.abs(f64(h) - want_h) <= ref.BF16 * np.abs(want_h) * 1.001 + rel * big * grow + rel * np.abs(want_h)).all()


@pytest.mark.parametrize("T, H", [(1, 8), (1, 64), (1, 2048), (1, 7168), (3, 1000), (5, 1032), (2, 4104), (1, 8192), (2, 16384), (2, 32768), (300, 8), (257, 264),
                                  (100, 520), (33, 1024), (2000, 2048), (129, 7168)])
@pytest.mark.parametrize("residual, gate, post, norm", [(None, "none", False, True), (torch.bfloat16, "none", False, True), (torch.float32, "token", True, True),
                                                        (torch.bfloat16, "channel", True, True), (torch.float32, "full", False, False)])
def test_sizes(T, H, residual, gate, post, norm):
    a = inputs(T, H, residual, gate, post, norm, T + H)
    r, h = fw.norm_residual(scale=0.75, **a)
    assert r.dtype == (residual or torch.bfloat16) and h.dtype == torch.bfloat16
    check(a, r, h, 0.75)


@pytest.mark.parametrize("gate", ["none", "channel", "channel16", "token", "token32", "full", "full32"])
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [640, 2048])
def test_gates(gate, residual, H):
    a = inputs(17, H, residual, gate, True, True)
    check(a, *fw.norm_residual(scale=-2.0, eps=1e-3, **a), scale=-2.0, eps=1e-3)


@pytest.mark.parametrize("T, H", [(1000, 1032), (700, 2048), (4097, 2560), (600, 5128), (999, 7168), (400, 8192), (310, 16384), (305, 32768)])
@pytest.mark.parametrize("residual, gate, post, norm, fp8", [(torch.bfloat16, "none", False, True, False), (torch.float32, "full32", True, True, False),
                                                             (None, "channel16", True, True, False), (torch.float32, "token", False, False, False),
                                                             (torch.bfloat16, "channel", False, True, True), (torch.bfloat16, "full", True, True, True)])
def test_many_rows(T, H, residual, gate, post, norm, fp8):
    """Rows enough that a CTA loops over several, in place too; the same as row by row in small calls."""
    fp8 = fp8 and H % 16 == 0
    a = inputs(T, H, residual, gate, post, norm, T + H)
    r, h = fw.norm_residual(scale=0.5, **a)
    some = [0, 1, 151, 152, 303, T - 2, T - 1]
    check({k: v[some] if v is not None and v.dim() == 2 and v.shape[0] == T else v for k, v in a.items()}, r[some], h[some], 0.5)
    part = {k: v[200:300] if v is not None and v.dim() == 2 and v.shape[0] == T else v for k, v in a.items()}
    r2, h2 = fw.norm_residual(scale=0.5, **part)
    u = ref.FP32 if residual is torch.float32 else ref.BF16
    near = lambda x, y, u: ((x.double() - y.double()).abs() <= 2.01 * u * y.double().abs() + 1e-4 * u * y.double().abs().amax(1, keepdim=True)).all()  # noqa: E731
    assert near(h[200:300], h2, ref.BF16) and (residual is torch.float32 or near(r[200:300], r2, u))
    if fp8:
        _, (codes, scales) = fw.norm_residual(scale=0.5, fp8=True, **a)
        want_c, want_s = fw.quantize_fp8(h)
        assert torch.equal(codes.view(torch.uint8), want_c.view(torch.uint8)) and torch.equal(scales, want_s)
    if residual is not None:
        into, out = a["residual"].clone(), a["y"].clone()
        b = dict(a, residual=into, y=out)
        fw.norm_residual(scale=0.5, residual_out=into, h=out, **b)
        assert torch.equal(into, r) and torch.equal(out, h)


@pytest.mark.parametrize("T, H", [(1, 16), (1, 2048), (4, 1040), (200, 144), (65, 7168), (3, 32768)])
def test_codes_are_those_of_the_bf16_result(T, H):
    a = inputs(T, H, torch.bfloat16, "channel", True, True)
    r, h = fw.norm_residual(**a)
    r8, (codes, scales) = fw.norm_residual(fp8=True, **a)
    want_c, want_s = fw.quantize_fp8(h)
    assert torch.equal(r, r8) and torch.equal(codes.view(torch.uint8), want_c.view(torch.uint8)) and torch.equal(scales, want_s)


def test_zeros_and_non_finite_rows_stay_in_their_rows():
    a = inputs(6, 512, torch.bfloat16, "none", True, True)
    a["y"][1], a["residual"][1] = 0, 0
    a["y"][2, 3] = float("inf")
    a["residual"][3, 9] = float("nan")
    a["y"][4] = 1e-30
    r, h = fw.norm_residual(**a)
    fine = [0, 1, 4, 5]
    part = {k: v[fine] if v is not None and v.dim() == 2 else v for k, v in a.items()}
    check(part, r[fine], h[fine])
    assert (h[1] == 0).all() and torch.isnan(h[2]).any() and torch.isnan(h[3]).all()


@pytest.mark.parametrize("T, H", [(5, 1024), (3, 2048)])
def test_views_and_in_place(T, H):
    a = inputs(T, H, torch.bfloat16, "full", True, True)
    want_r, want_h = fw.norm_residual(**a)
    wide = lambda t: torch.nn.functional.pad(t, (8, 24))[:, 8:8 + H]  # noqa: E731
    b = dict(a, y=wide(a["y"]), residual=wide(a["residual"]), gate=wide(a["gate"]))
    room = torch.full((T, H + 16), 5.0, dtype=torch.bfloat16, device=DEV)
    r, h = fw.norm_residual(residual_out=b["residual"], h=room[:, 8:8 + H], **b)
    assert r.data_ptr() == b["residual"].data_ptr()
    assert torch.equal(r, want_r) and torch.equal(h, want_h) and (room[:, :8] == 5).all() and (room[:, 8 + H:] == 5).all()
    r, h = fw.norm_residual(residual_out=a["residual"], h=a["y"], **a)
    assert torch.equal(r, want_r) and torch.equal(h, want_h)


def test_empty_streams_and_capture():
    a = inputs(9, 2048, torch.float32, "token", True, True)
    none = {k: v[:0] if v is not None and v.dim() == 2 else v for k, v in a.items()}
    r, h = fw.norm_residual(**none)
    assert r.shape == h.shape == (0, 2048)
    want = fw.norm_residual(**a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fw.norm_residual(stream=side.cuda_stream, **a)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fw.norm_residual(**a)
    a["y"].copy_(a["y"].flip(0))
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(got, fw.norm_residual(**a)))
