"""What the attention side's entry points say of a CUDA call that failed, and of sizes past their numbers."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import quantized_sparse_moe_router_gb300 as fw


@pytest.fixture(scope="module", autouse=True)
def built():
    fw.build()


def args(**over):
    a = dict(R=1, T=8, max_q=4, n_q=512, n_kv=4, D=128, page=16, n_pages=8, max_blocks=1 << 22, window=0, sinks=0, scale=0.1, q=4096, out=4096,
             q_stride=1 << 16, out_stride=1 << 16, cache=4096, block_table=4096, q_start=4096, seq_lens=4096, status=None)
    a.update(over)
    return ctypes.byref(fw.FwAttnQ4Args(**a))


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_no_device_is_named():
    need = ctypes.c_int64()
    assert fw.lib().fw_attn_q4_workspace(args(), ctypes.byref(need)) == fw.FW_ECUDA
    assert "cudaError" in fw.fw_moe_last_error()


def test_positions_that_pass_32_bits_when_rounded_up_are_refused():
    need = ctypes.c_int64()
    for page in (16, 128):
        few = dict(n_q=8, n_kv=1, page=page, max_blocks=(1 << 31) // page - 1)
        assert fw.lib().fw_attn_q4_workspace(args(**few), ctypes.byref(need)) == fw.FW_EINVAL and "max_blocks" in fw.fw_moe_last_error()


@pytest.mark.gpu
def test_a_launch_that_cannot_be_is_named_and_leaves_no_error_behind():
    """2^31 - 1 rows of q need more blocks than a grid has: nothing is launched, and none of these addresses is read."""
    assert fw.lib().fw_attn_q4(args(T=(1 << 31) - 1, max_q=(1 << 31) - 1), None, 0, torch.cuda.current_stream().cuda_stream) == fw.FW_ECUDA
    assert "fw_attn_q4: launch: cudaErrorInvalidValue" in fw.fw_moe_last_error()
    x = torch.ones(4, device="cuda")
    torch.cuda.synchronize()
    assert (x + x).sum().item() == 8
