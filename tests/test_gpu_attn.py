"""GPU parity of the attention side: the plan, the norms and rotation with the
store into the 4-bit cache, the read-back and the attention, against the plain
64-bit forms of attn_ref."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


# ------------------------------------------------------------------ plan
def run_plan(ctx, new, max_blocks, free, page, T_cap, used=0, stream=None):
    rng = np.random.default_rng(1)
    table = np.full((len(ctx), max_blocks), -1, np.int32)
    for r, c in enumerate(ctx):
        n = min(max_blocks, max(0, -(-c // page)))
        table[r, :n] = rng.integers(0, 1000, n) + 100
    t = ints(table) if len(ctx) else torch.zeros((0, max_blocks), dtype=torch.int32, device=DEV)
    p = fw.kv_plan(ints(ctx), ints(new), t, ints(free), page, T_cap, free_used=ints([used]) if used else None, stream=stream)
    torch.cuda.synchronize()
    want = ref.plan(ctx, new, table.tolist(), list(free), page, T_cap, used)
    got = [t.cpu().numpy().tolist()] + [x.cpu().numpy().tolist() for x in p]
    for g, w, name in zip(got, want, ("table",) + p._fields):
        assert g == w, name


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R", [1, 3, 64, 700, 2500])
def test_plan(R, page):
    rng = np.random.default_rng(R * page)
    ctx, new = rng.integers(0, 400, R).tolist(), rng.integers(0, 40, R).tolist()
    ctx[0], new[-1] = page, page + 1
    run_plan(ctx, new, -(-450 // page) + 1, rng.permutation(R * 60).tolist(), page, sum(new) + 7)


def test_plan_edges():
    run_plan([], [], 4, [1], 16, 5)                                   # no requests
    run_plan([0, 0, 0], [0, 0, 0], 4, [1], 16, 5)                     # nothing new
    run_plan([0], [1], 1, [9], 16, 1)                                 # one token
    run_plan([5, 16, 31], [11, 1, 2], 4, [9, 8, 7], 16, 14)           # a page filled to its end, opened, straddled
    run_plan([0], [5000], 400, list(range(400)), 16, 5000)            # one long request over several CTAs
    run_plan([3, 2], [40, 40], 4, list(range(20)), 16, 80, used=9)    # the free list in use from entry 9


def test_plan_reports():
    run_plan([0, 0], [40, 40], 4, [9, 8, 7], 16, 80)                  # the pool runs out
    run_plan([0, 30], [64, 40], 4, list(range(20)), 16, 104)          # a table row is full
    run_plan([0, 0], [40, 40], 4, list(range(20)), 16, 64)            # more tokens than places
    run_plan([-1, 2, 5, 4], [4, 3, -7, 2 ** 30], 4, list(range(20)), 16, 8)  # lengths that are none


def test_plan_continues_the_free_list():
    """Two steps in a row without the host: the second takes its free entries where the first stopped."""
    free, table = ints(range(100, 140)), ints(np.full((2, 8), -1))
    a = fw.kv_plan(ints([0, 0]), ints([20, 5]), table, free, 16, 32)
    b = fw.kv_plan(a.seq_lens, ints([20, 20]), table, free, 16, 64, free_used=a.counts[1:2])
    assert b.counts.tolist() == [40, 5, 0]
    assert table.cpu().tolist()[0][:3] == [100, 101, 103] and table.cpu().tolist()[1][:2] == [102, 104]
    s = b.slots.cpu().tolist()
    assert s[0] == 101 * 16 + 4 and s[12] == 103 * 16 and s[20] == 102 * 16 + 5 and s[31] == 104 * 16


# ------------------------------------------------------------------ norms, rotation, store
def rope_case(T, n_q, n_kv, D, rot, seed, norm=True, scale=1.0):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(scale * rng.standard_normal((T, (n_q + 2 * n_kv) * D))).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.to(DEV).split([n_q * D, n_kv * D, n_kv * D], 1))
    n_pos = 300
    ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))[None]
    cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    norms = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    return q, k, v, cos_sin, pos, norms


def check_rotated(got, x, norm, cos_sin, pos, interleaved):
    want, big = ref.rotate(x.double().cpu().numpy(), norm, 1e-6, cos_sin, np.maximum(pos, 0), interleaved)
    # one rounding to bf16, and fp32 sums of products of at most `big`: 16 roundings of 2^-24
    tol = ref.U * np.abs(want) * 1.001 + 2.0 ** -20 * big
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())


def on(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


@pytest.mark.parametrize("T, n_q, n_kv, D, rot, interleaved, norm", [
    (1, 32, 4, 128, 128, False, True), (1, 1, 1, 64, 64, False, True), (5, 3, 1, 64, 32, True, True), (33, 16, 16, 64, 16, False, False),
    (7, 14, 2, 128, 64, False, True), (2, 8, 1, 128, 128, True, False), (129, 5, 5, 128, 48, True, True), (3, 4, 2, 64, 0, False, True)])
def test_qk_norm_rope(T, n_q, n_kv, D, rot, interleaved, norm):
    q, k, _, cos_sin, pos, (qn, kn) = rope_case(T, n_q, n_kv, D, rot, T + D, norm)
    cs = on(cos_sin) if rot else torch.zeros((1, 0), device=DEV)
    qo, ko = fw.qk_norm_rope(q, k, on(pos), cs, on(qn), on(kn), interleaved=interleaved)
    check_rotated(qo, q, qn, cos_sin, pos, interleaved)
    check_rotated(ko, k, kn, cos_sin, pos, interleaved)


def test_qk_norm_rope_in_place_and_one_norm_only():
    q, k, _, cos_sin, pos, (qn, _) = rope_case(9, 8, 2, 128, 128, 3)
    q0, k0 = q.clone(), k.clone()
    qo, ko = fw.qk_norm_rope(q, k, on(pos), on(cos_sin), q_norm=on(qn), q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr()
    check_rotated(q, q0, qn, cos_sin, pos, False)
    check_rotated(k, k0, None, cos_sin, pos, False)


def test_qk_norm_rope_tiny_and_zero_rows():
    """Rows of zeros (the norm is eps alone) and values far from one."""
    for scale in (0.0, 1e-20, 1e18):
        q, k, _, cos_sin, pos, (qn, kn) = rope_case(4, 4, 2, 64, 64, 5, scale=scale)
        qo, ko = fw.qk_norm_rope(q, k, on(pos), on(cos_sin), on(qn), on(kn))
        check_rotated(qo, q, qn, cos_sin, pos, False)
        check_rotated(ko, k, kn, cos_sin, pos, False)


@pytest.mark.parametrize("T, n_q, n_kv, D, page, norm", [(1, 32, 4, 128, 16, True), (40, 8, 2, 64, 32, True), (129, 3, 3, 128, 64, False),
                                                         (300, 16, 1, 64, 128, True)])
def test_store_and_export(T, n_q, n_kv, D, page, norm):
    q, k, v, cos_sin, pos, (qn, kn) = rope_case(T, n_q, n_kv, D, D, T, norm)
    rng = np.random.default_rng(T)
    n_pages = -(-T // page) + 2
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    if T > 4:
        slots[2] = -1
        pos[2] = -1
    cache = fw.kv_cache(n_pages, n_kv, D, page)
    cache.fill_(0x5A)
    before = cache.clone()
    ko = torch.empty((T, n_kv, D), dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, _ = fw.qk_norm_rope(q, k, on(pos), on(cos_sin), on(qn), on(kn), v=v, cache=cache, slots=on(slots), k_out=ko, status=status)
    check_rotated(qo, q, qn, cos_sin, pos, False)
    check_rotated(ko, k, kn, cos_sin, pos, False)
    # the cache, byte for byte: the keys as rounded to bf16, and the values, by the block rule; no other byte written
    want = before.cpu().numpy()
    for x, which in ((ko, "k"), (v, "v")):
        c, d = ref.quantise(x.double().cpu().numpy())
        bits = ref.bf16_bits(d)
        for t in range(T):
            if slots[t] >= 0:
                for h in range(n_kv):
                    ref.write_block(want[slots[t] // page, h], page, D, slots[t] % page, which, c[t, h], bits[t, h])
    assert np.array_equal(cache.cpu().numpy(), want)
    ek, ev = fw.kv_export(cache, on(slots), D, status=status)
    for got, x in ((ek, ko), (ev, v)):
        c, d = ref.quantise(x.double().cpu().numpy())
        w = torch.from_numpy(ref.values(c, d).reshape(x.shape)).to(torch.bfloat16)
        w[torch.from_numpy(slots) < 0] = 0
        assert torch.equal(got.cpu(), w)
    assert status.item() == 0


def test_store_ties_extremes_and_non_finite_blocks():
    """Blocks whose extremes tie, all-zero blocks; a block with an infinity or
    NaN reads back as non-finite and leaves its neighbours alone."""
    D, page = 64, 16
    k = torch.zeros((4, 1, D), dtype=torch.bfloat16, device=DEV)
    k[0, 0, :2] = torch.tensor([-3.0, 3.0])
    k[1, 0, 5], k[1, 0, 40] = float("nan"), 2.0
    k[2, 0, 5], k[2, 0, 40] = float("inf"), -2.0
    v, q = k.clone(), torch.zeros((4, 1, D), dtype=torch.bfloat16, device=DEV)
    cache, slots = fw.kv_cache(1, 1, D, page), ints([3, 4, 5, 6])
    fw.qk_norm_rope(q, k, ints([0] * 4), torch.zeros((1, 0), device=DEV), v=v, cache=cache, slots=slots)
    for e in fw.kv_export(cache, slots, D):
        e = e.float().cpu()[:, 0]
        assert e[0, :3].tolist() == [-2.625, 3.0, 0.0] and not e[3].any()
        assert not torch.isfinite(e[1, :32]).any() and e[1, 40] == 2.0 and e[1, 32:].abs().sum() == 2.0
        assert not torch.isfinite(e[2, 5]) and e[2, 40] == -2.0 and e[2, 32:].abs().sum() == 2.0


@pytest.mark.parametrize("power", [0, -97, -120, 102, 110])
def test_store_every_quotient(power):
    """Codes are x / d rounded half to even for every pair of bf16 significands,
    at magnitudes around and past those where 1 / d is taken."""
    D, page = 128, 128
    x = np.zeros((128, 6, 5, 32))
    for y in range(128):
        for e in range(6):
            body = np.resize((128 + np.arange(128)) * 2.0 ** -e, (5, 31)) * np.where(np.arange(31) % 2, -1, 1)
            x[y, e, :, 1:] = np.where(np.abs(body) <= 128 + y, body, body / 2)
            x[y, e, :, 0] = (128 + y) * (1 if (y + e) % 2 else -1)
    v = torch.from_numpy(x.reshape(-1, 1, D) * 2.0 ** (power - 7)).to(torch.bfloat16)
    T = v.shape[0]
    cache, slots = fw.kv_cache(-(-T // page), 1, D, page), torch.arange(T, dtype=torch.int32, device=DEV)
    k = v.flip(0).contiguous().to(DEV)
    fw.qk_norm_rope(torch.zeros_like(k), k, torch.zeros_like(slots), torch.zeros((1, 0), device=DEV), v=v.to(DEV), cache=cache, slots=slots)
    want = np.zeros(tuple(cache.shape), np.uint8)
    for t in range(T):
        for which, w in (("k", k.cpu()), ("v", v)):
            c, d = ref.quantise(w[t].double().numpy())
            ref.write_block(want[t // page, 0], page, D, t % page, which, c[0], ref.bf16_bits(d)[0])
    assert np.array_equal(cache.cpu().numpy(), want)


def test_bad_slots_and_positions_are_reported_and_skipped():
    q, k, v, cos_sin, pos, _ = rope_case(4, 2, 1, 64, 64, 8)
    cache = fw.kv_cache(2, 1, 64, 16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos[1] = 300
    fw.qk_norm_rope(q, k, on(pos), on(cos_sin), v=v, cache=cache, slots=ints([0, 1, 32, -5]), status=status)
    assert status.item() == fw.KV_BAD_SLOT | fw.KV_BAD_POSITION
    status.zero_()
    e, _ = fw.kv_export(cache, ints([0, 32, -1]), 64, status=status)
    assert status.item() == fw.KV_BAD_SLOT and e[0].any() and not e[1:].any()


# ------------------------------------------------------------------ attention
def check_attn(case, window=0, sinks=0, scale=None, **kw):
    d = case.device()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], kw.pop("max_q", case.max_q), scale=scale,
                     window=window, sinks=sinks, status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, tol = case.reference(window, sinks, scale)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:5].tolist())
    return out


HEADS = [(8, 2, 128, 16), (4, 4, 64, 32), (16, 1, 128, 64), (14, 2, 64, 128), (5, 1, 128, 16)]


@pytest.mark.parametrize("n_q, n_kv, D, page", HEADS)
def test_attn_single_tokens(n_q, n_kv, D, page):
    check_attn(ref.Case([(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (128, 1), (129, 1), (300, 1), (1000, 1)], n_q, n_kv, D, page))


@pytest.mark.parametrize("n_q, n_kv, D, page", HEADS)
def test_attn_prompts(n_q, n_kv, D, page):
    check_attn(ref.Case([(40, 40), (1, 1), (130, 130), (300, 77), (257, 2)], n_q, n_kv, D, page, seed=1))


@pytest.mark.parametrize("new", [1, 2, 3, 4, 8, 17])
def test_attn_drafted_tokens(new):
    check_attn(ref.Case([(new, new), (333, new), (64, 1), (1500, new)], 8, 2, 128, 16, seed=new))


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (100, 4), (128, 17), (129, 200), (4000, 4)])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_attn_window(window, sinks, new):
    check_attn(ref.Case([(700, new), (new, new), (131, new), (90 + 5, min(new, 5))], 4, 2, 64, 16, seed=window), window, sinks)


def test_attn_no_requests_tokens_or_keys():
    """Requests without tokens, and a batch of only such."""
    check_attn(ref.Case([(0, 0), (50, 1), (70, 0), (3, 3), (0, 0)], 8, 2, 64, 16))
    c = ref.Case([(10, 0), (0, 0)], 8, 2, 64, 16)
    d = c.device()
    assert fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], 0).shape == (0, 8, 64)


@pytest.mark.parametrize("new", [3, 40])
def test_attn_rows_that_see_nothing_are_zero(new):
    """More new tokens than positions (a length not yet brought up to date): rows before position 0 see no key."""
    c = ref.Case([(2, 2), (100, new)], 8, 2, 128, 16)
    d = c.device()
    seq = d["seq_lens"].clone()
    seq[1] = new - 2
    out = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], seq, c.max_q).double().cpu().numpy()
    assert not out[2:4].any()
    k, v = c.k[1][:new - 2], c.v[1][:new - 2]
    want, tol = ref.attention(c.q.double().numpy()[2:], k, v, new, 1 / math.sqrt(128), 0, 0)
    assert (np.abs(out[2:] - want) <= tol).all()
    seq[1] = 0
    out = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], seq, c.max_q)
    assert not out[2:].any() and out[:2].any()


@pytest.mark.parametrize("new, window", [(1, 0), (1, 9), (4, 7), (200, 0), (200, 50)])
def test_attn_ignores_what_is_masked(new, window):
    """NaN in unused places of a page, in pages of nobody, and -- for a prompt --
    in keys and values that later rows see but earlier ones must not."""
    c = ref.Case([(210, new), (37, 1)], 8, 2, 128, 32, seed=2, fill=None)
    check_attn(c, window, 2 if window else 0)
    poison = 209  # the last position: seen by the last row only
    block = c.cache[c.table[0, poison // 32]]
    for h in range(2):
        for which in "kv":
            ref.write_block(block[h], 32, 128, poison % 32, which, np.full(128, 3), np.array([0x7FC0, 0x3F80, 0x7F80, 0x3F80]))
    d = c.device()
    out = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q, window=window, sinks=2 if window else 0)
    got = out.double().cpu().numpy()
    want, tol = c.reference(window, 2 if window else 0)
    assert (np.abs(got - want) <= tol)[:new - 1].all()      # rows that do not see it
    assert np.isnan(got[new - 1]).all()                      # the row that does: its score is NaN
    assert (np.abs(got - want) <= tol)[new:].all()           # the other request


@pytest.mark.parametrize("new", [1, 60])
def test_attn_infinite_value_reaches_only_rows_that_see_it(new):
    """A value block that is not finite makes the dims of its block NaN or infinite in the rows that see it, and no others."""
    c = ref.Case([(150, new)], 4, 1, 128, 16, seed=3)
    at = 149
    codes = np.full(128, 9)
    codes[0] = 8
    ref.write_block(c.cache[c.table[0, at // 16], 0], 16, 128, at % 16, "v", codes, np.array([0x7F80, 0x3F80, 0x3F80, 0x7FC0]))
    d = c.device()
    out = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q).double().cpu().numpy()
    want, tol = c.reference()
    assert (np.abs(out - want) <= tol)[:new - 1].all()
    assert not np.isfinite(out[new - 1][:, :32]).any() and np.isnan(out[new - 1][:, 96:]).all()
    assert np.isfinite(out[new - 1][:, 32:96]).all()


def test_attn_extreme_scores():
    """Scores far beyond fp32's exp range, both signs; one key holds all the weight."""
    check_attn(ref.Case([(300, 1), (140, 130)], 8, 2, 128, 16, seed=5, q_gain=1.5), scale=30.0)
    check_attn(ref.Case([(300, 1), (140, 130)], 8, 2, 128, 16, seed=5, q_gain=1.5), scale=1e-6)


@pytest.mark.parametrize("new, n_q", [(1, 8), (20, 4), (470, 8)])
@pytest.mark.parametrize("gains", [(1e-25, 0.0, 1.0, 1e30), (1e30, 1.0, 0.0, 1e-25), (0.0, 2.0 ** -30, 2.0 ** 30, 1e-3), (1e36, 1e36, 1e36, 1e36),
                                   (2.0 ** -110,) * 4])
def test_attn_values_of_any_magnitude(new, n_q, gains):
    """Values whose magnitude changes along the context, and by block of dims
    (whole tiles of zeros among them): each row is as exact as what it sees."""
    S, D, page = 480, 64, 32
    c = ref.Case([(S, new)], n_q, 1, D, page, seed=new)
    rng = np.random.default_rng(new)
    x = rng.standard_normal((S, 1, D)).clip(-3, 3) * np.repeat(gains, S // 4)[:, None, None] * np.repeat([1.0, 0.25], 32)
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    codes, d = ref.quantise(x)
    bits = ref.bf16_bits(d)
    for j in range(S):
        ref.write_block(c.cache[c.table[0, j // page], 0], page, D, j % page, "v", codes[j, 0], bits[j, 0])
    c.v[0] = ref.values(codes, d).reshape(S, 1, D)
    check_attn(c)


def test_attn_strided_and_into_out():
    c = ref.Case([(60, 1), (90, 30)], 8, 2, 64, 16, seed=6)
    d = c.device()
    wide = torch.full((c.T, 8 * 64 + 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :512] = d["q"].flatten(1)
    out_wide = torch.full((c.T, 8 * 64 + 128), 7.0, dtype=torch.bfloat16, device=DEV)
    out = fw.attn_q4(wide[:, :512].unflatten(1, (8, 64)), d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q,
                     out=out_wide[:, 64:576].unflatten(1, (8, 64)))
    want, tol = c.reference()
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert (out_wide[:, :64] == 7).all() and (out_wide[:, 576:] == 7).all()


def test_attn_more_rows_than_tokens_and_larger_max_q():
    """Rows of q past q_start[R] stay as they are, and max_q may be generous."""
    c = ref.Case([(60, 1), (90, 2)], 8, 2, 64, 16, seed=7)
    d = c.device()
    q = torch.cat([d["q"], torch.full((40, 8, 64), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out = torch.full_like(q, 5.0)
    fw.attn_q4(q, d["cache"], d["block_table"], d["q_start"], d["seq_lens"], 43, out=out)
    want, tol = c.reference()
    assert (np.abs(out[:3].double().cpu().numpy() - want) <= tol).all() and (out[3:] == 5).all()


@pytest.mark.parametrize("new", [1, 50])
def test_attn_bad_pages_are_reported_and_masked(new):
    c = ref.Case([(200, new), (100, 1)], 8, 2, 128, 16, seed=8)
    d = c.device()
    bt = d["block_table"].clone()
    bt[0, 1], bt[0, 4] = -1, c.cache.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fw.attn_q4(d["q"], d["cache"], bt, d["q_start"], d["seq_lens"], c.max_q, status=status).double().cpu().numpy()
    assert status.item() == fw.KV_BAD_SLOT
    j = np.arange(200)
    keep = (j // 16 != 1) & (j // 16 != 4)
    want, tol = ref.attention(c.q.double().numpy()[:new], c.k[0][keep], c.v[0][keep], new, 1 / math.sqrt(128), 0, 0)
    assert (np.abs(out[:new] - want) <= tol).all()
    want, tol = c.reference()
    assert (np.abs(out[new:] - want[new:]) <= tol[new:]).all()


@pytest.mark.parametrize("new", [1, 100])
def test_attn_same_bits_every_time_and_on_other_streams(new):
    c = ref.Case([(500, new), (100, 1), (30, min(new, 30))], 8, 2, 128, 16, seed=9)
    d = c.device()
    call = lambda **kw: fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q, **kw)  # noqa: E731
    first = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [call(stream=side.cuda_stream) for _ in range(8)]
    with torch.cuda.stream(side):
        got += [call() for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, g) for g in got)


@pytest.mark.parametrize("n_q, n_kv, D, page, new", [(8, 8, 64, 16, 1), (16, 4, 128, 64, 1), (8, 4, 128, 32, 5), (32, 2, 128, 128, 1)])
def test_attn_many_segments_many_calls(n_q, n_kv, D, page, new):
    """Many more 128-key units than CTAs, so that a CTA takes several heads and
    requests in a row, and many calls without a wait between them."""
    rng = np.random.default_rng(n_q)
    c = ref.Case([(int(s), new) for s in rng.integers(new, 2600 if D == 128 else 1200, 60)], n_q, n_kv, D, page, seed=4)
    first = check_attn(c)
    d = c.device()
    args = (d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q)
    got = [fw.attn_q4(*args) for _ in range(200)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, g) for g in got)


def test_attn_long_contexts():
    """A few long contexts: many units in a row of one head, split over many CTAs."""
    check_attn(ref.Case([(20000, 1), (9000, 2), (13001, 1)], 8, 2, 128, 128, seed=12))


def many_blocks(D, page, n_q=16, n_kv=2, seed=21):
    """Prompts and chunks of several 256-row blocks, the last ones of 128 rows and
    fewer among them, with single tokens and short drafts in between."""
    new = [290, 261, 33, 16, 300, 1, 272, 250, 10, 288, 299, 230, 303, 2, 281]
    past = [0, 130, 500, 3, 0, 700, 17, 128, 260, 1, 0, 511, 64, 9, 390]
    return ref.Case([(n + s, n) for n, s in zip(new, past)], n_q, n_kv, D, page, seed=seed)


@pytest.mark.parametrize("D, page, window, sinks", [(64, 16, 0, 0), (128, 64, 0, 0), (64, 128, 70, 3), (128, 32, 200, 0)])
def test_attn_many_blocks(D, page, window, sinks):
    c = many_blocks(D, page)
    first = check_attn(c, window, sinks)
    d = c.device()
    for _ in range(20):
        got = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q, window=window, sinks=sinks)
    assert torch.equal(got, first)


def test_attn_many_blocks_infinite_value():
    """The only rows that a value block that is not finite reaches are those of its request and head at its position or after."""
    c = many_blocks(64, 32, seed=22)
    r, at, head = 4, 150, 1
    want, tol = c.reference()
    ref.write_block(c.cache[c.table[r, at // 32], head], 32, 64, at % 32, "v", np.full(64, 9), np.array([0x7F80, 0x3F80]))
    d = c.device()
    out = fw.attn_q4(d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q).double().cpu().numpy()
    hit = np.zeros(out.shape, bool)
    hit[c.starts[r] + at:c.starts[r + 1], 8 * head:8 * head + 8] = True
    assert (np.abs(out - want) <= tol)[~hit].all()
    assert not np.isfinite(out[hit].reshape(-1, 64)[:, :32]).any() and np.isfinite(out[hit].reshape(-1, 64)[:, 32:]).all()


def test_attn_in_a_cuda_graph():
    c = ref.Case([(500, 1), (100, 1), (300, 40)], 8, 2, 128, 16, seed=10)
    d = c.device()
    out = torch.empty_like(d["q"])
    args = (d["cache"], d["block_table"], d["q_start"], d["seq_lens"], c.max_q)
    fw.attn_q4(d["q"], *args, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fw.attn_q4(d["q"], *args, out=out)
    first = out.clone()
    out.zero_()
    d["q"].mul_(1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)


def test_attn_python_refusals():
    c = ref.Case([(60, 1)], 8, 2, 64, 16)
    d = c.device()
    args = [d["q"], d["cache"], d["block_table"], d["q_start"], d["seq_lens"], 1]
    for i, bad in ((0, d["q"].half()), (0, d["q"].transpose(1, 2)), (1, d["cache"].int()), (1, d["cache"][..., :-8].contiguous()),
                   (2, d["block_table"].long()), (2, d["block_table"][:, ::2]), (3, d["q_start"][:1]), (4, d["seq_lens"].cpu())):
        with pytest.raises(ValueError):
            fw.attn_q4(*[bad if k == i else a for k, a in enumerate(args)])
    with pytest.raises(fw.FwError):
        fw.attn_q4(*args, window=-1)
