"""Pages whose bytes lie past 2^32 in the cache, for the store, the read-back and each form of the attention."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw
from attn_cases import DEV, unpacked_ahead

pytestmark = pytest.mark.gpu


def far_cache(pages, n_kv, D, page, seed=0):
    """A cache past 4.5 GB with the given pages (uint8 [n, ...]) at the end of it, in another order -> cache, their ids."""
    size = n_kv * ref.page_bytes(page, D)
    n = 4_500_000_000 // size + len(pages)
    assert n * page < 2 ** 31
    ids = n - 1 - np.random.default_rng(seed).permutation(len(pages))
    cache = torch.zeros((n, n_kv, size // n_kv), dtype=torch.uint8, device=DEV)
    assert int(ids.min()) * size > 2 ** 32
    cache[torch.from_numpy(ids).to(DEV)] = torch.from_numpy(pages).to(DEV)
    return cache, ids


@pytest.mark.parametrize("lens, n_q, n_kv, D, page, ahead", [
    ([(700, 1), (333, 2)], 8, 2, 128, 16, False), ([(700, 60), (500, 90)], 8, 4, 64, 128, False), ([(300, 220)], 96, 12, 64, 32, True)])
def test_attention_past_4_gb(lens, n_q, n_kv, D, page, ahead):
    c = ref.Case(lens, n_q, n_kv, D, page, seed=1)
    assert unpacked_ahead(c) == ahead
    cache, ids = far_cache(c.cache, n_kv, D, page)
    table = np.where(c.table >= 0, ids[c.table], -1).astype(np.int32)
    d = c.device()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fw.attn_q4(d["q"], cache, torch.from_numpy(table).to(DEV), d["q_start"], d["seq_lens"], c.max_q, status=status)
    want, tol = c.reference()
    assert status.item() == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_store_and_read_back_past_4_gb():
    n_kv, D, page, T = 2, 128, 16, 40
    cache, ids = far_cache(np.zeros((5, n_kv, ref.page_bytes(page, D)), np.uint8), n_kv, D, page)
    slots = torch.from_numpy((np.repeat(ids, 8) * page + np.tile(np.arange(8), 5)).astype(np.int32)).to(DEV)
    rng = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(T, h, D, generator=rng, device=DEV).bfloat16() for h in (4, n_kv, n_kv))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    fw.qk_norm_rope(q, k, torch.zeros_like(slots), torch.zeros((1, 0), device=DEV), v=v, cache=cache, slots=slots, status=status)
    for got, x in zip(fw.kv_export(cache, slots, D, status=status), (k, v)):
        codes, d = ref.quantise(x.double().cpu().numpy())
        assert torch.equal(got.cpu(), torch.from_numpy(ref.values(codes, d).reshape(x.shape)).to(torch.bfloat16))
    assert status.item() == 0
    near = cache[:(1 << 20) // cache.shape[1]]  # (where 32 bits would have put them)
    assert not near.any()
