"""Routing rules set on another stream than the current one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import synth
from layer_inputs import DeviceLayer, to_device_bf16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("then", ["another bias", "no bias", "the default step"])
def test_a_bias_lasts_until_its_copy(then):
    """A rule, a route and another rule wait on a stream that is held up, while the first rule's bias is let go of and
    the current stream makes and fills tensors of its size."""
    E, k, T = 64, 4, 8
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV)
    layer = dl.make(T_max=T)
    x = to_device_bf16(synth.hidden_bf16_bits(w, 0), DEV)
    raise_ = lambda first: torch.from_numpy(np.where((np.arange(E) >= first) & (np.arange(E) < first + k), 4.0, 0.0).astype(np.float32)).to(DEV)  # noqa: E731
    want = [list(range(20, 20 + k))] * T
    chosen = lambda ids: ids.sort(1).values.tolist()  # noqa: E731
    layer.set_routing("sigmoid", bias=raise_(20))  # (the first rule allocates)
    assert chosen(layer.route(x)[0]) == want
    layer.set_routing("sigmoid")
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    bias, other = raise_(20), raise_(40)
    side = torch.cuda.Stream()
    fill = lambda: [torch.full((E,), 9.0 * (i % 2), device=DEV) for i in range(64)]  # noqa: E731
    fill()  # (its kernel is loaded before the other stream sleeps)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some 0.2 s
    layer.set_routing("sigmoid", bias=bias, stream=side.cuda_stream)
    layer.route(x, expert_ids=ids, stream=side.cuda_stream)
    if then == "another bias":
        layer.set_routing("sigmoid", bias=other, stream=side.cuda_stream)
    elif then == "no bias":
        layer.set_routing("sigmoid", stream=side.cuda_stream)
    else:
        layer.set_routing(None)
    del bias
    filled = fill()
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # (it was still held up: the test shows something)
    torch.cuda.synchronize()
    assert len(filled) == 64 and chosen(ids) == want
    layer.close()
