"""Calls on another stream than the current one: the memory that they make for
themselves is none that the current stream's queued work still uses."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw
from attn_cases import workspace

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def plan():
    R, T_cap = 300, 1 << 20
    ctx, new, table, free = ints([5] * R), ints([9] * R), ints(np.full((R, 4), 7)), ints(np.arange(R))
    return lambda **kw: fw.kv_plan(ctx, new, table, free, 16, T_cap, **kw), [4 * (3 * T_cap + 2 * R + 4)]


def rope():
    T = 3000
    q, k = (torch.ones((T, h, 64), dtype=torch.bfloat16, device=DEV) for h in (8, 3))
    pos, cos_sin = ints(np.zeros(T)), torch.zeros((1, 64), device=DEV)
    return lambda **kw: fw.qk_norm_rope(q, k, pos, cos_sin, **kw), [T * 8 * 128, T * 3 * 128]


def export():
    cache, slots = fw.kv_cache(50, 5, 64, 128), ints(np.arange(6000))
    return lambda **kw: fw.kv_export(cache, slots, 64, **kw), [6000 * 5 * 256]


def attention():
    c = ref.Case([(2000, 900)], 8, 2, 128, 16)
    d = c.device()
    assert workspace(c) > 1 << 20
    return (lambda **kw: fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q, **kw),
            [900 * 8 * 256, workspace(c)])


@pytest.mark.parametrize("made", [plan, rope, export, attention])
def test_memory_of_another_streams_call_is_not_the_current_streams(made):
    call, sizes = made()
    side = torch.cuda.Stream()
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
    del got


def test_results_of_another_streams_call_may_be_used_on_the_current_one():
    """A result freed while the current stream still reads it is not given to the other stream's next call."""
    call, _ = rope()
    side = torch.cuda.Stream()
    first, _ = call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    want, to = first.clone(), torch.zeros_like(first)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    to.copy_(first)
    del first
    with torch.cuda.stream(side):
        others = [torch.full((3000, 8, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(to, want)
    del others
