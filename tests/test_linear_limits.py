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


class Tensor:
    """What the calls ask a tensor for, of a shape that no memory holds."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, shape, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def get_device(self):
        return 0


@pytest.mark.parametrize("shape", [((1 << 32) + 5, 16), (1 << 31, 16), (3, 1 << 32), (1, (1 << 31) + 16)])
def test_sizes_past_32_bits_are_refused(shape):
    """(Passed on, they would be cut to 32 bits: 2^32 + 5 tokens to 5.)"""
    with pytest.raises(ValueError, match="2\\^31"):
        fw.quantize_fp8(Tensor(torch.bfloat16, *shape))
    with pytest.raises(ValueError, match="2\\^31"):
        fw.quantize_fp8_weight(Tensor(torch.bfloat16, *shape))
