"""Host-side checks of the attention side's torch calls."""
import pytest

torch = pytest.importorskip("torch")

import quantized_sparse_moe_router_gb300 as fw
from quantized_sparse_moe_router_gb300 import attention


class On:
    """A tensor as far as its device goes."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("devices, current, ok", [((0, 0, 0), 0, True), ((1, 1), 1, True), ((0, 1), 0, False), ((1, 0), 0, False), ((1, 1), 0, False)])
def test_tensors_have_to_be_on_the_current_device(monkeypatch, devices, current, ok):
    monkeypatch.setattr(attention, "_several", True)
    monkeypatch.setattr(attention, "_current_device", lambda: current)
    tensors = [On(d) for d in devices] + [None]
    if ok:
        attention._one_device("call", *tensors)
    else:
        with pytest.raises(ValueError, match="current device"):
            attention._one_device("call", *tensors)


@pytest.mark.gpu
def test_calls_refuse_tensors_of_another_device(monkeypatch):
    """Each call asks, before it makes or launches anything."""
    ints = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, q = fw.kv_cache(2, 1, 64, 16), torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    calls = [lambda: fw.kv_plan(ints(0), ints(1), ints(0, 0)[None], ints(0, 1), 16, 4),
             lambda: fw.qk_norm_rope(q, q, ints(0), torch.zeros((1, 64), device="cuda")),
             lambda: fw.kv_export(cache, ints(0), 64),
             lambda: fw.attn_q4(q, cache, ints(0, 1)[None], ints(0, 1), ints(1), 1)]
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
