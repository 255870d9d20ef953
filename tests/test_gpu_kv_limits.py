"""The plan and the store at the limits of their numbers."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import quantized_sparse_moe_router_gb300 as fw

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [16, 128])
def test_page_ids_past_every_cache(page):
    """Page ids whose slots would pass 32 bits, in the table and in the free list:
    their tokens' slots are no cache's, and a store reports and skips them."""
    wraps = 2 ** 32 // page  # times the page: 0 in 32 bits
    table = ints([[wraps, -1], [2 ** 31 - 1, -1], [0, -1], [-1, -1]])
    p = fw.kv_plan(ints([1, 1, 1, 0]), ints([1, 1, 1, 2]), table, ints([wraps // 2]), page, 5)
    top = 2 ** 31 - 1
    assert p.slots.tolist() == [top, top, 1, top, top]
    cache = fw.kv_cache(3, 1, 64, page)
    k = torch.ones((5, 1, 64), dtype=torch.bfloat16, device="cuda")
    status = ints([0])
    fw.qk_norm_rope(k.clone(), k, p.positions, torch.zeros((1, 0), device="cuda"), v=k, cache=cache, slots=p.slots, status=status)
    assert status.item() == fw.KV_BAD_SLOT
    got, _ = fw.kv_export(cache, ints([0, 1, 2]), 64)
    assert got.float().sum(2).flatten().tolist() == [0.0, 64.0, 0.0]
