"""Host-side checks of the 8-bit linear layers and the norms at the residual
stream: bad arguments are refused before any CUDA call, nothing to do is no error."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp8_ref as ref
import quantized_sparse_moe_router_gb300 as fw


@pytest.fixture(scope="module", autouse=True)
def built():
    fw.build()


def call_quantize(**over):
    a = dict(x=4096, x_stride=256, T=3, K=256, codes=4096, scales=4096, scale_stride=4)
    a.update(over)
    return fw.lib().fw_fp8_quantize(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(K=0), dict(K=24), dict(x=None), dict(codes=None), dict(scales=None), dict(x_stride=248), dict(x_stride=260),
                                 dict(x=4104), dict(codes=4104), dict(scales=4104), dict(scale_stride=3), dict(scale_stride=0), dict(scale_stride=6)])
def test_quantize_refuses(bad):
    assert call_quantize(**bad) == fw.FW_EINVAL and fw.fw_moe_last_error()


@pytest.mark.parametrize("bad", [dict(N=0), dict(K=8), dict(K=-16), dict(w_fp32=2), dict(w=None), dict(codes=None), dict(scales=None), dict(w=4100), dict(codes=4097),
                                 dict(N=(1 << 31) - 1, K=(1 << 31) - 128)])
def test_quantize_weight_refuses(bad):
    a = dict(w=4096, w_fp32=1, N=64, K=256, codes=4096, scales=4096)
    a.update(bad)
    if torch.cuda.is_available() or "N" not in bad or bad["N"] == 0:  # (too many blocks: asked after the device)
        assert fw.lib().fw_fp8_quantize_weight(*a.values(), None) == fw.FW_EINVAL and fw.fw_moe_last_error()


def linear_args(**over):
    a = dict(T=40, K=256, N=64, out_fp32=0, x=4096, x_scale=None, x_stride=256, x_scale_stride=40, w=4096, w_scale=4096, out=4096, out_stride=64, status=None)
    a.update(over)
    return ctypes.byref(fw.FwLinearFp8Args(**a))


@pytest.mark.parametrize("bad, status", [(dict(T=-1), -1), (dict(K=0), -1), (dict(K=120), -1), (dict(N=0), -1), (dict(out_fp32=2), -1), (dict(T=(1 << 22) + 1), -4),
                                         (dict(N=(1 << 26) + 1), -4)])
def test_linear_refuses_sizes(bad, status):
    need = ctypes.c_int64(7)
    assert fw.lib().fw_linear_fp8_workspace(linear_args(**bad), ctypes.byref(need)) == status and need.value == 0
    assert fw.lib().fw_linear_fp8(linear_args(**bad), None, 0, None) == status and fw.fw_moe_last_error()


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(w_scale=None), dict(out=None), dict(x=4104), dict(w=4104), dict(x_scale=4104), dict(x_scale=4096, x_scale_stride=36), dict(x_scale=4096, x_scale_stride=42), dict(out=4097),
                                 dict(out=4098, out_fp32=1), dict(x_stride=248), dict(x_stride=260), dict(x_scale=4096, x_stride=264), dict(out_stride=63),
                                 dict(status=4098)])
def test_linear_refuses_pointers(bad):
    assert fw.lib().fw_linear_fp8(linear_args(**bad), 65536, 1 << 40, None) == fw.FW_EINVAL and fw.fw_moe_last_error()


def test_linear_workspace():
    need = ctypes.c_int64()
    assert fw.lib().fw_linear_fp8_workspace(linear_args(T=300, K=400, x_stride=400), ctypes.byref(need)) == fw.FW_OK
    assert need.value >= 300 * 400 + 4 * 300 * 4
    for at, size in ((None, 1 << 30), (4096, need.value - 1), (4104, 1 << 30)):
        assert fw.lib().fw_linear_fp8(linear_args(T=300, K=400, x_stride=400), at, size, None) == fw.FW_EINVAL
        assert "workspace" in fw.fw_moe_last_error()
    assert fw.lib().fw_linear_fp8_workspace(linear_args(T=300, x_scale=4096, x_scale_stride=300), ctypes.byref(need)) == fw.FW_OK and need.value == 0
    assert fw.lib().fw_linear_fp8_workspace(linear_args(), None) == fw.FW_EINVAL


def norm_args(**over):
    a = dict(T=3, H=256, residual_fp32=0, gate_fp32=0, gate_per_token=0, eps=1e-6, scale=1.0, y=4096, residual=4096, gate=4096, y_stride=256, residual_stride=256,
             gate_stride=256, post_norm=4096, norm=4096, residual_out=4096, h=4096, residual_out_stride=256, h_stride=256, h_codes=4096, h_scale=4096, h_scale_stride=4)
    a.update(over)
    return ctypes.byref(fw.FwNormResidualArgs(**a))


@pytest.mark.parametrize("bad, status", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(H=12), -1), (dict(H=32776), -4), (dict(H=264, y_stride=264), -1), (dict(residual_fp32=2), -1), (dict(gate_fp32=-1), -1),
    (dict(gate_per_token=3), -1), (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(y=None), -1), (dict(h_scale=None), -1),
    (dict(residual_out=None, h=None, h_codes=None), -1), (dict(y_stride=248), -1), (dict(y_stride=260), -1), (dict(residual_stride=8), -1),
    (dict(residual_out_stride=252), -1), (dict(h_stride=255), -1), (dict(gate_stride=128), -1), (dict(gate_stride=257), -1),
    (dict(gate_per_token=1, gate_stride=-1), -1), (dict(y=4104), -1), (dict(residual=4100), -1), (dict(gate=4104), -1), (dict(norm=4100), -1),
    (dict(post_norm=4104), -1), (dict(residual_out=4098), -1), (dict(h=4100), -1), (dict(h_codes=4104), -1), (dict(h_scale=4104), -1), (dict(h_scale_stride=2), -1), (dict(h_scale_stride=5), -1),
    (dict(gate_per_token=1, gate=4097), -1)])
def test_norm_residual_refuses(bad, status):
    assert fw.lib().fw_norm_residual(norm_args(**bad), None) == status and fw.fw_moe_last_error()


def test_nothing_to_do():
    assert call_quantize(T=0, x=None) == fw.FW_OK
    assert fw.lib().fw_linear_fp8(linear_args(T=0, x=None), None, 0, None) == fw.FW_OK
    assert fw.lib().fw_norm_residual(norm_args(T=0, y=None), None) == fw.FW_OK
    assert fw.lib().fw_linear_fp8(None, None, 0, None) == fw.FW_EINVAL
    assert fw.lib().fw_norm_residual(None, None) == fw.FW_EINVAL


def test_structs_match_the_header(tmp_path):
    """ctypes lays the argument structs out as a C compiler does the header's."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    by = {"fw_linear_fp8_args": fw.FwLinearFp8Args, "fw_norm_residual_args": fw.FwNormResidualArgs}
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "fwmoe.h"\nint main(void) {\n'
    for s, c in by.items():
        src += "".join(f'printf("%zu\\n", offsetof({s}, {n}));\n' for n, _ in c._fields_) + f'printf("%zu\\n", sizeof({s}));\n'
    (tmp_path / "a.c").write_text(src + "return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")], check=True)
    got = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [v for c in by.values() for v in [getattr(c, n).offset for n, _ in c._fields_] + [ctypes.sizeof(c)]]


def test_packed_arguments_are_the_structs():
    """What the torch calls pack is what ctypes makes of the same values, field by field."""
    from quantized_sparse_moe_router_gb300 import linear
    for pack, kind in ((linear._linear_args, fw.FwLinearFp8Args), (linear._norm_args, fw.FwNormResidualArgs)):
        values = list(range(3, 3 + len(kind._fields_)))
        assert pack(*values) == bytes(kind(*values))


@pytest.mark.parametrize("call", [lambda t: fw.quantize_fp8(t), lambda t: fw.quantize_fp8_weight(t), lambda t: fw.linear_fp8(t, t, t), lambda t: fw.norm_residual(t)])
def test_torch_calls_refuse_host_tensors(call):
    with pytest.raises(ValueError):
        call(torch.zeros(2, 256, dtype=torch.bfloat16))


def test_reference_of_the_codes():
    """The reference's codes: every value to itself, ties to even, and torch's own conversion."""
    assert np.array_equal(ref.encode(ref.VALUES), np.arange(127)) and ref.VALUES[126] == 448
    assert ref.encode([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 460.0, -0.0]).tolist() == [0x38, 0x3A, 0, 2, 126, 0x80]
    x = np.concatenate([np.random.default_rng(0).normal(size=20000) * s for s in (0.01, 1.0, 100.0)]).astype(np.float32).clip(-448, 448)
    assert np.array_equal(ref.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_of_a_block():
    """m, scale and codes of a block by hand: m = 2 -> scale 2 / 448; 1 -> 224, an eighth of m's step below it rounds there."""
    x = np.zeros((1, 16))
    x[0, :3] = 2.0, -1.0, 0.0078125
    c, s = ref.quantise(x, 1)
    assert s[0, 0] == np.float32(2) / np.float32(448)
    assert ref.decode(c)[0, :4].tolist() == [448.0, -224.0, 1.75, 0.0]
