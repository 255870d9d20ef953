"""Hidden values that round up to the next power of two when they are brought to 16 bits, in the fused expert kernel."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_sparse_moe_router_gb300 as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
H, I, E = 128, 64, 4


def blocks(scales, codes):
    """fp16 [R, C / 32] and int8 [R, C] -> Q8_0 bytes."""
    R, C = codes.shape
    b = np.zeros((R, C // 32, 34), np.uint8)
    b[:, :, :2] = scales.astype(np.float16).reshape(R, C // 32, 1).view(np.uint8)
    b[:, :, 2:] = codes.reshape(R, C // 32, 32).view(np.uint8)
    return b.reshape(-1)


def just_below():
    """Scales g, u with 127 g >= 17 (its SiLU is itself to 2^-24) and 127^2 g u below 32 by 2^-17 to 2^-20 of it."""
    g = np.arange(0x3000 + 0x060, 0x3400, dtype=np.uint16).view(np.float16).astype(np.float64)  # from 0.137 on
    u = np.arange(0x1C00, 0x2C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    off = 1.0 - 127.0 ** 2 * g[:, None] * u[None] / 32.0
    at = np.argwhere((off > 2.0 ** -20) & (off < 2.0 ** -17) & (127 * g[:, None] >= 17))
    return g[at[0, 0]], u[at[0, 1]]


@pytest.mark.parametrize("T", [1, 2, 16])
@pytest.mark.parametrize("sign", [1, -1])
def test_just_below_a_power_of_two(T, sign):
    rng = np.random.default_rng(5)
    g, u = just_below()
    gate, up = np.zeros((I, H), np.int8), np.zeros((I, H), np.int8)
    gate[:, 0] = 127
    up[:, 0] = rng.integers(-60, 60, I)
    up[::16, 0] = sign * 127  # the largest of each 16, just below 32
    down = rng.integers(-127, 128, (H, I)).astype(np.int8)
    wg, wu, wd = (blocks(np.full((c.shape[0], c.shape[1] // 32), s), c) for s, c in ((g, gate), (u, up), (0.01, down)))
    stack = lambda b: torch.from_numpy(np.stack([b] * E)).to(DEV)  # noqa: E731
    moe = fw.MoELayer(H, I, E, 1, T_max=16, weights=dict(router_w=torch.randn(E, H, device=DEV), w_gate=stack(wg), w_up=stack(wu), w_down=stack(wd)))
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1.0
    out = moe.forward(x)[1].double().cpu().numpy()
    moe.status()
    moe.close()
    a, b = 127.0 * g, up[:, 0].astype(np.float64) * u
    h = a / (1.0 + np.exp(-a)) * b
    want = (down.astype(np.float64) * float(np.float16(0.01))) @ h
    # out is rounded to bf16; h to 2^-15 of the largest of its 16
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * np.abs(down.astype(np.float64) * 0.01) @ np.repeat(np.abs(h).reshape(-1, 16).max(1), 16)
    assert (np.abs(out - want) <= tol * 1.01).all()
