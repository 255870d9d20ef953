"""The example's decoder layer: plan, norms and rotation with the store,
attention and the routed experts in one step, against the plain 64-bit forms."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("window, sinks", [(0, 0), (40, 4)])
def test_attention_of_each_step(window, sinks):
    """Prompts, single tokens and drafts over the cache that the steps before filled."""
    layer = ex.DecoderLayer(window=window, sinks=sinks)
    req = ex.Requests(3, layer, page=16, n_pages=64)
    g = torch.Generator(device="cuda").manual_seed(3)
    held = [([], []) for _ in range(3)]  # keys and values as the cache holds them
    past = [0, 0, 0]
    for new in ((70, 1, 33), (1, 1, 1), (1, 40, 0), (4, 2, 3)):
        T = sum(new)
        x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
        lens = torch.tensor(new, dtype=torch.int32, device="cuda")
        plan = fw.kv_plan(req.lens, lens, req.block_table, req.free_pages, req.page, T, free_used=req.used)
        out = f64(layer.attend(x, plan, req.cache, req.block_table, max(new), req.status))
        req.lens.copy_(plan.seq_lens)
        req.used.copy_(plan.counts[1:2])
        assert req.status.item() == 0 and plan.counts[2].item() == 0
        q, k, v = layer.project(x)
        q, k = fw.qk_norm_rope(q, k, plan.positions, layer.cos_sin, layer.q_norm, layer.k_norm)
        pos = plan.positions.cpu().numpy()
        for got, raw, norm in ((q, layer.project(x)[0], layer.q_norm), (k, layer.project(x)[1], layer.k_norm)):
            want, big = ref.rotate(f64(raw), f64(norm), 1e-6, layer.cos_sin.cpu().numpy(), pos, False)
            # one rounding to bf16, and 16 of 2^-24 of the largest value
            assert (np.abs(f64(got) - want) <= ref.U * np.abs(want) * 1.001 + 2.0 ** -20 * big).all()
        at = 0
        for r, n in enumerate(new):
            for which, t in ((0, k), (1, v)):
                held[r][which].append(ref.values(*ref.quantise(f64(t[at:at + n]))).reshape(n, layer.n_kv, layer.D))
            past[r] += n
            K, V = (np.concatenate(h) for h in held[r])
            want, tol = ref.attention(f64(q[at:at + n]), K, V, n, layer.D ** -0.5, window, sinks)
            assert (np.abs(out[at:at + n] - want) <= tol).all()
            at += n
    assert req.lens.tolist() == past


def test_example():
    """Piece by piece (prompts, a replayed graph, drafts) against whole requests.
    Both see the same 4-bit keys and values; what differs is the rounding to
    bf16 of a few sums, except where a token's second and third expert are as
    good as tied."""
    layer = ex.DecoderLayer()
    pieces, whole, cached = ex.run(layer)
    assert cached.lens.tolist() == [p.shape[0] for p in pieces]
    for a, b in zip(pieces, whole):
        a, b = f64(a), f64(b)
        assert np.isfinite(a).all()
        rows = np.abs(a - b).max(1)
        # 16 roundings of bf16 at the row's largest value
        near = rows <= 16 * ref.U * np.abs(b).max(1)
        assert near.mean() >= 0.95, (float(rows.max()), float(near.mean()))
