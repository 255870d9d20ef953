"""Attention where the key tiles are unpacked ahead of it (six row blocks of 256
and more a request, enough of them for all SMs): the same properties that the
other attention tests check where tiles are not."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw
from attn_cases import DEV, call, check, set_values, unpacked_ahead

pytestmark = pytest.mark.gpu


def prompt(S, new, D=64, page=32, G=8, n_kv=12, seed=0, **kw):
    """One request of `new` tokens; twelve key heads make its blocks enough for the SMs."""
    c = ref.Case([(S, new)], G * n_kv, n_kv, D, page, seed=seed, **kw)
    assert unpacked_ahead(c)
    return c


def several(D, page, seed=21):
    """Prompts and chunks with single tokens, short drafts and an empty request in between."""
    new = [420, 1, 460, 3, 0, 401, 700, 2]
    past = [0, 300, 77, 64, 50, 260, 1, 5]
    c = ref.Case([(n + s, n) for n, s in zip(new, past)], 32, 4, D, page, seed=seed)
    return c


@pytest.mark.parametrize("S, new, D, page, G, n_kv", [(200, 200, 64, 16, 8, 12), (517, 230, 128, 32, 8, 12), (300, 111, 64, 128, 16, 11),
                                                      (1601, 1601, 128, 64, 1, 11), (385, 385, 128, 16, 4, 11)])
def test_ahead_prompts(S, new, D, page, G, n_kv):
    check(prompt(S, new, D, page, G, n_kv, seed=S))


@pytest.mark.parametrize("D, page, window, sinks", [(64, 16, 0, 0), (128, 64, 0, 0), (64, 128, 70, 3), (128, 32, 200, 0), (128, 16, 128, 129)])
def test_ahead_several_requests_and_many_calls(D, page, window, sinks):
    c = several(D, page)
    assert unpacked_ahead(c, window, sinks)
    check(c, window, sinks)
    d = c.device()
    args = (d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q)
    got = [fw.attn_q4(*args, window=window, sinks=sinks) for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, got[0]) for g in got)


@pytest.mark.parametrize("window, sinks", [(1, 0), (5, 3), (100, 4), (128, 17), (129, 200), (4000, 4)])
def test_ahead_window(window, sinks):
    c = prompt(430, 220, seed=window)
    assert unpacked_ahead(c, window, sinks)
    check(c, window, sinks)


@pytest.mark.parametrize("window", [0, 50])
def test_ahead_ignores_what_is_masked(window):
    """NaN in unused places of a page, in pages of nobody and in the last position, which one row sees."""
    c = prompt(210, 205, 128, 32, seed=2, fill=None)
    block = c.cache[c.table[0, 209 // 32]]
    for h in range(c.n_kv):
        for which in "kv":
            ref.write_block(block[h], 32, 128, 209 % 32, which, np.full(128, 3), np.array([0x7FC0, 0x3F80, 0x7F80, 0x3F80]))
    got = call(c, window, 2 if window else 0)
    want, tol = c.reference(window, 2 if window else 0)
    assert (np.abs(got - want) <= tol)[:-1].all() and np.isnan(got[-1]).all()


def test_ahead_infinite_value_reaches_only_rows_that_see_it():
    c = prompt(400, 300, seed=22)
    at, head = 350, 5
    want, tol = c.reference()
    ref.write_block(c.cache[c.table[0, at // 32], head], 32, 64, at % 32, "v", np.full(64, 9), np.array([0x7F80, 0x3F80]))
    out = call(c)
    hit = np.zeros(out.shape, bool)
    hit[at - 100:, 8 * head:8 * head + 8] = True
    assert (np.abs(out - want) <= tol)[~hit].all()
    assert not np.isfinite(out[hit].reshape(-1, 64)[:, :32]).any() and np.isfinite(out[hit].reshape(-1, 64)[:, 32:]).all()


def test_ahead_bad_pages_are_reported_and_masked():
    c = prompt(330, 215, 128, 16, seed=8)
    table = c.table.copy()
    table[0, 1], table[0, 12] = -1, c.cache.shape[0]
    out = call(c, table=table, status=fw.KV_BAD_SLOT)
    keep = ~np.isin(np.arange(330) // 16, (1, 12))
    want = np.zeros(out.shape)
    tol = np.zeros(out.shape)
    for i in range(215):  # a position's place among the keys that are left is not its number
        see = keep & (np.arange(330) <= 115 + i)
        w, t = ref.attention(c.q.double().numpy()[i:i + 1], c.k[0][see], c.v[0][see], 1, 1 / math.sqrt(128), 0, 0)
        want[i], tol[i] = w[0], t[0]
    assert (np.abs(out - want) <= tol).all()


def test_ahead_extreme_scores():
    c = prompt(300, 210, seed=5)
    check(c, scale=30.0)
    check(c, scale=1e-6)


def test_ahead_in_a_cuda_graph_and_on_another_stream():
    c = prompt(260, 230, 128, 64, seed=10)
    d = c.device()
    out = torch.empty_like(d["q"])
    args = (d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q)
    fw.attn_q4(d["q"], *args, out=out)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fw.attn_q4(d["q"], *args, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    side = torch.cuda.Stream()
    got = [fw.attn_q4(d["q"], *args, stream=side.cuda_stream) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, x) for x in got)


GAINS = [(0.0, 1.0, 1.0, 1.0), (0.0, 0.05, 0.05, 0.05), (0.0, 1e-3, 1e-3, 0.0), (0.0, 2.0 ** -30, 2.0 ** -30, 2.0 ** -30), (1e-3,) * 4,
         (1e-25, 0.0, 1.0, 1e30), (1e30, 1.0, 0.0, 1e-25), (0.0, 2.0 ** -30, 2.0 ** 30, 1e-3), (1e30,) * 4, (2.0 ** -110,) * 4]


def magnitudes(gain, seed):
    """A prompt whose values have the size gain[j] at position j."""
    S = len(gain)
    c = prompt(S, 210, seed=seed)
    rng = np.random.default_rng(seed)
    set_values(c, 0, rng.standard_normal((S, c.n_kv, 64)).clip(-3, 3) * np.asarray(gain)[:, None, None] * np.repeat([1.0, 0.25], 32))
    return c


@pytest.mark.parametrize("gains", GAINS)
def test_ahead_values_of_any_magnitude(gains):
    """Values whose magnitude changes along the context, whole tiles of zeros among them."""
    check(magnitudes(np.repeat(gains, 128), 7))


@pytest.mark.parametrize("small, rest", [(1e-6, 1.0), (1e-6, 0.05), (1e-6, 0.01), (1e3, 1e-3), (1e6, 0.01)])
def test_ahead_one_block_of_another_size(small, rest):
    """One position of the first tile whose values have another size than all others."""
    gain = np.full(500, rest)
    gain[3] = small
    check(magnitudes(gain, 8))


@pytest.mark.parametrize("first, low, high", [(2.0 ** 41, 2.0 ** 20, 2.0 ** 60), (2.0 ** 30, 1.0, 2.0 ** 30), (2.0 ** 30, 2.0 ** -20, 1.0)])
def test_ahead_a_tile_of_very_unequal_values_after_large_ones(first, low, high):
    """A tile of large values, then tiles whose values differ among themselves by
    up to 2^40: what counts is what each row gives weight to."""
    gain = np.full(512, first)
    gain[128:] = np.where(np.arange(384) % 5, low, high)
    check(magnitudes(gain, 9))


def test_ahead_rows_that_do_not_see_the_large_values():
    """Large values at the last position of the second tile: only rows from there on see them, and later tiles are small again."""
    gain = np.full(400, 0.02)
    gain[255] = 2.0 ** 30
    check(magnitudes(gain, 10))
