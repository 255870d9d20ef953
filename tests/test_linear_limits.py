"""Sizes next to and past what 32 bits hold, in the calls of the 8-bit linear layers, without a device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import quantized_sparse_moe_router_gb300 as fw

LAST = (1 << 31) - 16  # the largest K: a multiple of 16


@pytest.mark.parametrize("K", [LAST, (1 << 31) - 128, (1 << 31) - 112, 1 << 30])
def test_workspace_of_the_largest_k(K):
    """Codes of 17 tokens, and scales of ceil(K / 128) blocks of them."""
    fw.build()
    args, need = fw.FwLinearFp8Args(T=17, K=K, N=1, x_stride=K, out_stride=1), ctypes.c_int64()
    assert fw.lib().fw_linear_fp8_workspace(ctypes.byref(args), ctypes.byref(need)) == fw.FW_OK
    assert need.value >= 17 * K + 4 * 17 * -(-K // 128)

