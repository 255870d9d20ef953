"""The example's layer in 8 bits: norms, linear layers, attention's store and the ruled experts in one step, each stage against
the plain 64-bit form of what it was given."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import fp8_ref as ref
import quantized_sparse_moe_router_gb300 as fw
import rule_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def check_linear(y, codes, scales, w):
    """y against the sums over these codes: the sums' own error, and one rounding to bf16."""
    want, tol = ref.linear(bits(codes), f64(scales).T, bits(w[0]), f64(w[1]))
    assert (np.abs(f64(y) - want) <= tol + ref.BF16 * (np.abs(want) + tol)).all()


def check_norm(got, y, residual, norm, post):
    want_r, want_h, big = ref.norm_residual(f64(y), f64(residual), None if norm is None else f64(norm), f64(post), None, 1.0, 1e-6)
    fp = (y.shape[1] / 2 + 8) * ref.FP32  # (as in the norms' own tests)
    assert (np.abs(f64(got[0]) - want_r) <= ref.BF16 * np.abs(want_r) * 1.001 + fp * big).all()
    if norm is not None:
        grow = np.abs(f64(norm)) / np.sqrt((want_r ** 2).mean(1, keepdims=True) + 1e-6)
        assert (np.abs(f64(got[1]) - want_h) <= ref.BF16 * np.abs(want_h) * 1.001 + 2 * fp * (big * grow + np.abs(want_h))).all()


def test_stages_of_each_step():
    """Prompts, single tokens and drafts; the step as one call has the bits of its stages."""
    layer = ex.EightBitLayer()
    req = ex.Requests(3, layer, page=16, n_pages=64)
    g = torch.Generator(device="cuda").manual_seed(3)
    for new in ((70, 1, 33), (1, 1, 1), (1, 40, 0), (4, 2, 3)):
        T = sum(new)
        x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
        lens = torch.tensor(new, dtype=torch.int32, device="cuda")
        plan = fw.kv_plan(req.lens, lens, req.block_table, req.free_pages, req.page, T, free_used=req.used)
        codes, scales = fw.norm_residual(x, norm=layer.norm1, fp8=True)[1]
        h = fw.norm_residual(x, norm=layer.norm1)[1]
        # the codes are of the norm before its rounding to bf16: a scale's rounding and half a step of a code, 2^-4 of
        # the value (2^-10 of the block's scale at least), beside that rounding
        want = f64(h)
        block = np.repeat(f64(scales).T, 128, 1)[:, :512]
        got = ref.values(bits(codes), f64(scales).T, 1)
        assert (np.abs(got - want) <= (2.0 ** -4 + 2 * ref.BF16) * np.abs(want) * 1.01 + 2.0 ** -10 * block * 1.01).all()
        y = torch.cat(layer.project(x), 1).reshape(T, -1)
        check_linear(y, codes, scales, layer.qkv8)
        o = layer.attend(x, plan, req.cache, req.block_table, max(new), req.status)
        rows = o.view(T, -1)
        a = fw.linear_fp8(rows, *layer.o8)
        check_linear(a, *fw.quantize_fp8(rows), layer.o8)
        r, h = layer.join(x, o)
        check_norm((r, h), a, x, layer.norm2, layer.post1)
        ids, out = layer.moe.forward(h)
        z = f64(h) @ f64(layer.router).T
        rule = dict(layer.rule, bias=f64(layer.rule["bias"]))
        choice, _, far = rule_ref.choose(z, 4, **rule)
        clear = far > 1e-4
        assert clear.mean() > 0.9 and np.array_equal(ids.cpu().numpy()[clear], choice[clear])
        y = fw.norm_residual(out, r, post_norm=layer.post2)
        check_norm(y, out, r, None, layer.post2)
        again = layer.forward(x, plan, req.cache, req.block_table, max(new), req.status)  # (the same keys and values into the same places)
        assert torch.equal(again.view(torch.int16), y[0].view(torch.int16))
        req.lens.copy_(plan.seq_lens)
        req.used.copy_(plan.counts[1:2])
        assert req.status.item() == 0 and plan.counts[2].item() == 0
    layer.moe.status()


def test_example():
    """It runs: prompts, a replayed graph and drafts, and whole requests. (Sums of other tile shapes differ in their last bits,
    and a code of 8 bits by a step where one was near a tie: a few of a row's codes, 2^-4 each of values that add up at random,
    so most rows are much nearer than a tenth.)"""
    layer = ex.EightBitLayer()
    pieces, whole, cached = ex.run(layer)
    assert cached.lens.tolist() == [p.shape[0] for p in pieces]
    for a, b in zip(pieces, whole):
        a, b = f64(a), f64(b)
        assert np.isfinite(a).all() and np.isfinite(b).all()
        rel = np.linalg.norm(a - b, axis=1) / np.linalg.norm(b, axis=1)
        assert np.median(rel) <= 0.1
