"""The attention side of a served layer, next to its routed experts: the cases that are measured, and each operator's plain form.

Three operators over a paged cache that holds keys and values in 4 bits:

  plan  block tables, slot map and positions of a step, from the requests' lengths
  qkv   norms of queries and keys for each head with the position rotation, and keys and values stored into the cache
  attn  causal attention of a step's new tokens over that cache (optionally a sliding window with first tokens that stay visible)

Page format (one page of P tokens of one key/value head, D dims, NB = D / 32 blocks; P * D * 9 / 8 bytes):
  K codes  [P][4 q][NB b] words of 32 bits: dims 32 b + 8 q + {0, 2, 4, 6, 1, 3, 5, 7} in nibbles 0..7
  K scales [P][NB] bf16
  V codes  [P / 2][8 g][NB b] words: dims 32 b + 4 g + {0, 1, 2, 3} of the even token in nibbles 0..3, of the odd token in 4..7
  V scales [P / 2][NB][2] bf16, the even token's and the odd token's
A value is scale * (code - 8); a block's scale is its element of largest magnitude (of two, the positive one) over -8.
"""
import math
import random

import torch

own = False

DEV = "cuda"
PHI = 0.6180339887498949


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of a busy server: one token for each of 64 requests
        dict(name="plan_decode", op="plan", R=64, ctx_min=1, ctx_max=8191, new_min=1, new_max=1, page=16),
        # many prompts admitted at once, some with a cached prefix
        dict(name="plan_prompts", op="plan", R=509, ctx_min=0, ctx_max=1023, new_min=1, new_max=900, page=64),
        # one user's next token, stored into the cache
        dict(name="qkv_token", op="qkv", T=1, n_q=32, n_kv=4, D=128, rot=128, interleaved=False, norm=True, store=True, page=16),
        # a middling batch, interleaved partial rotation, no norms, no cache
        dict(name="qkv_partial", op="qkv", T=257, n_q=16, n_kv=16, D=64, rot=32, interleaved=True, norm=False, store=False, page=16),
        # a prompt chunk stored into the cache
        dict(name="qkv_prompt", op="qkv", T=4096, n_q=32, n_kv=4, D=128, rot=128, interleaved=False, norm=True, store=True, page=64),
        # one user's next token after about a thousand: latency
        dict(name="attn_token", op="attn", R=1, n_q=32, n_kv=4, D=128, page=16, ctx_min=1000, ctx_max=1000, new_min=1, new_max=1, window=0, sinks=0),
        # a decode step of a busy server, ragged contexts
        dict(name="attn_batch", op="attn", R=64, n_q=32, n_kv=4, D=128, page=64, ctx_min=100, ctx_max=8191, new_min=1, new_max=1, window=0, sinks=0),
        # a few very long contexts
        dict(name="attn_long", op="attn", R=4, n_q=32, n_kv=4, D=128, page=128, ctx_min=98304, ctx_max=131071, new_min=1, new_max=1, window=0, sinks=0),
        # four drafted tokens checked at once by windowed layers with kept first tokens
        dict(name="attn_draft_window", op="attn", R=48, n_q=16, n_kv=4, D=64, page=16, ctx_min=0, ctx_max=16383, new_min=1, new_max=4, window=1024, sinks=4),
        # one prompt from nothing
        dict(name="attn_prompt", op="attn", R=1, n_q=32, n_kv=4, D=128, page=64, ctx_min=0, ctx_max=0, new_min=4096, new_max=4096, window=0, sinks=0),
        # chunks of a few prompts on top of what is cached, of odd lengths
        dict(name="attn_chunks", op="attn", R=3, n_q=32, n_kv=4, D=128, page=16, ctx_min=2000, ctx_max=9000, new_min=333, new_max=2047, window=0, sinks=0),
        # prompts through windowed layers, small heads, one head to each key head
        dict(name="attn_prompt_window", op="attn", R=2, n_q=8, n_kv=8, D=64, page=32, ctx_min=0, ctx_max=500, new_min=2500, new_max=4000, window=512, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "qkv", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "plan":
        new = _log(rng, 1, 900)
        return dict(op="plan", R=_log(rng, 1, 509), ctx_min=0, ctx_max=_log(rng, 1, 8191), new_min=rng.randint(0, min(new, 1)), new_max=new, page=page)
    D = rng.choice([64, 128])
    n_q, n_kv = rng.choice([(32, 4), (16, 4), (8, 8), (16, 2), (8, 1), (32, 8), (14, 2), (16, 1)])
    if kind == "qkv":
        return dict(op="qkv", T=_log(rng, 1, 4096), n_q=n_q, n_kv=n_kv, D=D, rot=rng.choice([32, 64, D]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                    store=rng.random() < 0.6, page=page)
    window, sinks = (0, 0) if rng.random() < 0.6 else (_log(rng, 1, 4096), rng.choice([0, 1, 4, 17]))
    if rng.random() < 0.6:  # single tokens, or a few drafted ones
        ctx = _log(rng, 1, 131071)
        R = _log(rng, 1, max(1, min(64, 262144 // ctx)))
        new = rng.choice([1, 1, 1, 2, 4])
    else:  # prompts
        new = _log(rng, 17, 2047)
        ctx = _log(rng, 1, 8191)
        R = _log(rng, 1, max(1, min(8, 4000000 // (new * (ctx + new)))))
    return dict(op="attn", R=R, n_q=n_q, n_kv=n_kv, D=D, page=page, ctx_min=rng.randint(0, ctx), ctx_max=ctx, new_min=rng.randint(1, new), new_max=new, window=window, sinks=sinks)


def _spread(lo, hi, n, start):
    """n whole numbers between lo and hi, spread evenly over the range."""
    return [lo + int((hi - lo + 1) * ((start + i * PHI) % 1.0)) for i in range(n)]


def _lengths(case):
    """(cached, new) lengths of the requests; the seed only sets their order."""
    return _spread(case["ctx_min"], case["ctx_max"], case["R"], 0.999), _spread(case["new_min"], case["new_max"], case["R"], 0.777)


def _visible(first, n, window, sinks):
    """(pairs, keys): the keys that queries at positions first .. first + n - 1 see, summed, and how many keys any of them sees."""
    if not window:
        return n * first + n * (n + 1) // 2, first + n
    lo = max(0, first + 1 - window)
    pairs = sum(min(p + 1, min(window, p + 1) + min(sinks, max(0, p + 1 - window))) for p in range(first, first + n))
    return pairs, (first + n - lo) + min(sinks, lo)


def work(case):
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        pages = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(ctx, new))
        return {"bytes": 4 * (2 * case["R"] + 2 * case["R"] + 2 * pages + 3 * sum(new)), "flops": 0}
    D, n_q, n_kv = case["D"], case["n_q"], case["n_kv"]
    if case["op"] == "qkv":
        T = case["T"]
        heads = 2 * n_q + (4 if case["store"] else 2) * n_kv  # q, k (and v) read; q and k (and v's and k's values) written
        return {"bytes": T * (2 * D * heads + 4 * case["rot"] + 8 + (2 * n_kv * D * 9 // 16 if case["store"] else 0)), "flops": T * (n_q + n_kv) * D * 8}
    ctx, new = _lengths(case)
    seen = [_visible(c, n, case["window"], case["sinks"]) for c, n in zip(ctx, new)]
    pairs, keys = sum(p for p, _ in seen), sum(k for _, k in seen)
    return {"bytes": keys * n_kv * D * 9 // 8 + sum(new) * n_q * D * 4, "flops": 4 * D * n_q * pairs}


# ------------------------------------------------------------------ the 4-bit blocks, as torch operations
def _quantise(x):
    """[..., D] bf16 -> codes 0..15 (uint8, [..., D]) and scales (bf16, [..., D / 32])."""
    b = x.float().unflatten(-1, (-1, 32))
    high, low = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
    d = torch.where(high >= -low, high, low) / -8.0  # exact in bf16: the element itself is
    q = torch.where(d != 0, torch.round(b / d), torch.zeros_like(b)) + 8.0
    return q.clamp(0, 15).to(torch.uint8).flatten(-2), d.squeeze(-1).to(torch.bfloat16)


def _values(codes, scales):
    return ((codes.float() - 8.0).unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)


def _pack_k(codes):
    """[..., D] codes -> [..., D / 2] bytes of K."""
    n = codes.dim() - 1
    c = codes.unflatten(-1, (-1, 4, 2, 2, 2))  # b, q, j / 2, j % 2, parity of the dim
    c = c.permute(*range(n), n + 1, n, n + 4, n + 2, n + 3)
    return (c[..., 0] | (c[..., 1] << 4)).flatten(n)


def _unpack_k(raw):
    n = raw.dim() - 1
    c = torch.stack((raw & 15, raw >> 4), -1).unflatten(n, (4, -1, 2, 2))  # q, b, parity, j / 2, j % 2
    return c.permute(*range(n), n + 1, n, n + 3, n + 4, n + 2).flatten(n)


def _pack_v(codes):
    """[..., D] codes of one token -> [..., D / 4, 2] bytes: its half of the words of its pair."""
    n = codes.dim() - 1
    c = codes.unflatten(-1, (-1, 8, 2, 2)).permute(*range(n), n + 1, n, n + 2, n + 3)  # g, b, j / 2, j % 2
    return (c[..., 0] | (c[..., 1] << 4)).flatten(n, n + 1)


def _unpack_v(raw):
    n = raw.dim() - 2
    c = torch.stack((raw & 15, raw >> 4), -1).unflatten(n, (8, -1))  # g, b, j / 2, j % 2
    return c.transpose(n, n + 1).flatten(n)


def _planes(cache, page, D):
    """Views of the four planes of [n_pages, n_kv, bytes]: K codes [.., page, D/2], K scales [.., page, NB], V codes [.., page/2, D/4, 2 tokens, 2], V scales [.., page/2, NB, 2]."""
    kc, ks = page * D // 2, page * (D // 32) * 2
    k, sk, v, sv = cache[..., :kc], cache[..., kc:kc + ks], cache[..., kc + ks:2 * kc + ks], cache[..., 2 * kc + ks:]
    return (k.unflatten(-1, (page, D // 2)), sk.unflatten(-1, (page, -1)), v.unflatten(-1, (page // 2, D // 4, 2, 2)), sv.unflatten(-1, (page // 2, -1, 2, 2)))


def _store(cache, page, D, slots, k_codes, k_scales, v_codes, v_scales):
    """Writes the tokens' blocks ([T, n_kv, ...]) to their slots; slots of -1 write nothing."""
    at = torch.div(slots, page, rounding_mode="floor").long()
    t = (slots % page).long()
    kc, ks, vc, vs = _planes(cache, page, D)
    kc[at, :, t] = _pack_k(k_codes)
    ks[at, :, t] = k_scales.view(torch.uint8)
    vc[at, :, t // 2, :, t % 2] = _pack_v(v_codes)
    vs[at, :, t // 2, :, t % 2] = v_scales.unsqueeze(-1).view(torch.uint8)


def _load(cache, page, D):
    """Keys and values of [..., n_kv, bytes] as fp32 [..., n_kv, page, D]."""
    kc, ks, vc, vs = _planes(cache, page, D)
    k = _values(_unpack_k(kc), ks.contiguous().view(torch.bfloat16))
    v = _values(_unpack_v(vc.movedim(-2, -3)).flatten(-3, -2),
                vs.contiguous().view(torch.bfloat16).squeeze(-1).transpose(-1, -2).flatten(-3, -2))
    return k, v


# ------------------------------------------------------------------ inputs
def _order(seed, R):
    order = list(range(R))
    random.Random(seed).shuffle(order)
    return order


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    page = case["page"]
    s = dict(case)
    if case["op"] == "qkv":
        T, n_q, n_kv, D, rot = case["T"], case["n_q"], case["n_kv"], case["D"], case["rot"]
        qkv = normal(T, (n_q + 2 * n_kv) * D).to(torch.bfloat16)  # the projection's output
        q, k, v = qkv.split([n_q * D, n_kv * D, n_kv * D], dim=1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (n_q, D)), k.unflatten(1, (n_kv, D)), v.unflatten(1, (n_kv, D))
        s["q_norm"], s["k_norm"] = (1.0 + 0.1 * normal(D), 1.0 + 0.1 * normal(D)) if case["norm"] else (None, None)
        n_pos = 8192
        angle = torch.arange(n_pos, device=DEV)[:, None] * (10000.0 ** (-torch.arange(0, rot, 2, device=DEV) / rot))[None, :]
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        first = random.Random(seed).randrange(n_pos - T)
        s["positions"] = torch.arange(first, first + T, dtype=torch.int32, device=DEV)
        if case["store"]:
            n_pages = -(-T // page) + 3
            at = torch.randperm(n_pages, generator=g, device=DEV)
            t = torch.arange(T, device=DEV) + page // 2
            s["slots"] = (at[t // page] * page + t % page).int()
            s["cache"] = torch.zeros(n_pages, n_kv, page * D * 9 // 8, dtype=torch.uint8, device=DEV)
        return s
    ctx, new = _lengths(case)
    order = _order(seed, case["R"])
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    total = [c + n for c, n in zip(ctx, new)]
    need = [-(-t // page) for t in (ctx if case["op"] == "plan" else total)]
    blocks = max(-(-t // page) for t in total)
    n_pages = sum(-(-t // page) for t in total) + 5
    at = torch.randperm(n_pages, generator=g, device=DEV).int()
    rows = torch.tensor(need, device=DEV)[:, None]
    before = torch.cumsum(rows, 0) - rows
    cols = torch.arange(blocks, device=DEV)[None, :]
    s["block_table"] = torch.where(cols < rows, at[(before + cols).clamp(max=n_pages - 1)], torch.full_like(at[:1], -1)).contiguous()
    if case["op"] == "plan":
        s["ctx"], s["new"], s["free_pages"], s["T_cap"] = _ints(ctx), _ints(new), at[sum(need):].contiguous(), -(-max(1, sum(new)) // 64) * 64
        return s
    n_q, n_kv, D = case["n_q"], case["n_kv"], case["D"]
    s["cache"] = torch.empty(n_pages, n_kv, page * D * 9 // 8, dtype=torch.uint8, device=DEV)
    for i in range(0, n_pages, 4096 * 16 // page):  # a stretch of pages at a time, to bound what the quantiser holds
        part = s["cache"][i:i + 4096 * 16 // page]
        slots = torch.arange(part.shape[0] * page, device=DEV)
        k, v = (_quantise(normal(slots.numel(), n_kv, D).to(torch.bfloat16)) for _ in range(2))
        _store(part, page, D, slots, *k, *v)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["q"] = (1.5 * normal(start[-1], n_q, D)).to(torch.bfloat16)
    s["q_start"], s["seq_lens"], s["max_q"] = _ints(start), _ints(total), max(new)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_plan(s):
    page, T, table = s["page"], s["T_cap"], s["block_table"]
    ctx, new = s["ctx"].long(), s["new"].long()
    total = ctx + new
    have, need = (ctx + page - 1) // page, (total + page - 1) // page
    taken = torch.cumsum(need - have, 0)
    cols = torch.arange(table.shape[1], device=DEV)[None, :]
    fresh = (cols >= have[:, None]) & (cols < need[:, None])
    index = (taken - (need - have))[:, None] + cols - have[:, None]
    table = torch.where(fresh, s["free_pages"][index.clamp(0, s["free_pages"].numel() - 1)], table)
    start = torch.cat((torch.zeros_like(taken[:1]), torch.cumsum(new, 0)))
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(start[1:], t, right=True)
    valid = r < new.numel()
    r = r.clamp(max=new.numel() - 1)
    pos = ctx[r] + t - start[r]
    slot = table[r, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    none = torch.full_like(t, -1)
    out = [torch.where(valid, x, none).int() for x in (r, pos, slot)]
    counts = torch.stack((start[-1], taken[-1], torch.zeros_like(taken[-1]))).int()
    return [table, start.int(), total.int(), *out, counts]


def _plain_norm_rope(x, w, s):
    y = x.float()
    if w is not None:
        y = y * (1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6)) * w
    rot = s["rot"]
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if s["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((r, y[..., rot:]), -1).to(torch.bfloat16)


def _plain_qkv(s):
    q, k = _plain_norm_rope(s["q"], s["q_norm"], s), _plain_norm_rope(s["k"], s["k_norm"], s)
    if not s["store"]:
        return [q, k]
    k, v = _quantise(k), _quantise(s["v"])
    _store(s["cache"], s["page"], s["D"], s["slots"], *k, *v)
    return [q, _values(*k).to(torch.bfloat16), _values(*v).to(torch.bfloat16)]


def _plain_attn(s):
    R, n_q, n_kv, D, page, most = s["R"], s["n_q"], s["n_kv"], s["D"], s["page"], s["max_q"]
    start, seq = s["q_start"].long(), s["seq_lens"].long()
    k, v = _load(s["cache"][s["block_table"].clamp(min=0).long()], page, D)  # [R, blocks, n_kv, page, D]
    k, v = k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)  # [R, n_kv, L, D]
    i = torch.arange(most, device=DEV)[None, :]
    n = (start[1:] - start[:-1])[:, None]
    q = s["q"].float()[(start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]  # [R, most, n_q, D]
    q = q.unflatten(2, (n_kv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, n_kv, most * G, D]
    p = (seq[:, None] - n + i)[..., None]  # positions [R, most, 1]
    j = torch.arange(k.shape[2], device=DEV)
    see = (j <= p) & (i < n)[..., None]
    if s["window"]:
        see &= (j > p - s["window"]) | (j < s["sinks"])
    see = see.repeat_interleave(n_q // n_kv, 1)[:, None]  # [R, 1, most * G, L]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).masked_fill_(~see, -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.unflatten(2, (most, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R, most, n_q, D]
    t = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(start[1:], t, right=True)
    return [out[r, t - start[r]].to(torch.bfloat16)]


def run(s):
    if not own:
        return {"plan": _plain_plan, "qkv": _plain_qkv, "attn": _plain_attn}[s["op"]](s)
    import quantized_sparse_moe_router_gb300 as fw
    if s["op"] == "plan":
        p = fw.kv_plan(s["ctx"], s["new"], s["block_table"], s["free_pages"], s["page"], s["T_cap"])
        return [s["block_table"], p.q_start, p.seq_lens, p.requests, p.positions, p.slots, p.counts]
    if s["op"] == "attn":
        return [fw.attn_q4(s["q"], s["cache"], s["block_table"], s["q_start"], s["seq_lens"], s["max_q"], window=s["window"], sinks=s["sinks"])]
    norms = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], interleaved=s["interleaved"])
    if not s["store"]:
        return list(fw.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], **norms))
    q, _ = fw.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], v=s["v"], cache=s["cache"], slots=s["slots"], **norms)
    return [q, *fw.kv_export(s["cache"], s["slots"], s["D"])]


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_plan(s):
    ctx, new, free, page = s["ctx"].tolist(), s["new"].tolist(), s["free_pages"].tolist(), s["page"]
    table, start, req, pos, slot, used = s["block_table"].tolist(), [0], [], [], [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        for b in range(-(-c // page), -(-(c + n) // page)):
            table[r][b] = free[used]
            used += 1
        start.append(start[-1] + n)
        req += [r] * n
        pos += range(c, c + n)
        slot += [table[r][p // page] * page + p % page for p in range(c, c + n)]
    pad = [-1] * (s["T_cap"] - start[-1])
    return [_ints(x) for x in (table, start, [c + n for c, n in zip(ctx, new)], req + pad, pos + pad, slot + pad, [start[-1], used, 0])]


def _exact_rotated(x, w, s):
    x = x.double()
    if w is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
    rot, out = s["rot"], x.clone()
    turn = torch.complex(*s["cos_sin"].double()[s["positions"].long()].split(rot // 2, 1))[:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_held(x):
    """What a 4-bit block stands for, of bf16 values."""
    b = x.to(torch.bfloat16).double().reshape(*x.shape[:-1], -1, 32)
    d = -torch.where(b.amax(-1) >= -b.amin(-1), b.amax(-1), b.amin(-1)).unsqueeze(-1) / 8
    return (torch.where(d == 0, 0.0, b / d).round().clamp(-8, 7) * d).reshape(x.shape)


def _exact_word(cache, at, head, byte):
    """Bytes of the cache at page `at`, by flat index, as whole numbers."""
    return cache.view(-1)[(at * cache.shape[1] + head) * cache.shape[2] + byte].to(torch.int32)


def _exact_scale(cache, at, head, byte):
    bits = _exact_word(cache, at, head, byte) | (_exact_word(cache, at, head, byte + 1) << 8)
    return (bits << 16).view(torch.float32).double()


def _exact_kv(cache, pages, head, n, page, D):
    """Keys and values of one head at positions 0 .. n - 1, one byte at a time from the format."""
    nb = D // 32
    j = torch.arange(n, device=DEV)
    at, t, d = pages[j // page].long()[:, None], (j % page)[:, None], torch.arange(D, device=DEV)[None, :]
    b, q, i = d // 32, d % 32 // 8, d % 8
    nib = i // 2 + 4 * (i % 2)
    code = (_exact_word(cache, at, head, t * (D // 2) + (q * nb + b) * 4 + nib // 2) >> (4 * (nib % 2))) & 15
    k = (code - 8).double() * _exact_scale(cache, at, head, page * D // 2 + (t * nb + b) * 2)
    base, g, i = page * D // 2 + page * nb * 2, d % 32 // 4, d % 4
    nib = i + 4 * (t % 2)
    code = (_exact_word(cache, at, head, base + (t // 2) * D + (g * nb + b) * 4 + nib // 2) >> (4 * (nib % 2))) & 15
    v = (code - 8).double() * _exact_scale(cache, at, head, base + page * D // 2 + ((t // 2) * nb + b) * 4 + (t % 2) * 2)
    return k, v


def _exact_attn(s):
    start, seq = s["q_start"].tolist(), s["seq_lens"].tolist()
    G = s["n_q"] // s["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for r in range(s["R"]):
        n = start[r + 1] - start[r]
        for h in range(s["n_kv"]):
            k, v = _exact_kv(s["cache"], s["block_table"][r], h, seq[r], s["page"], s["D"])
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                q = s["q"][start[r] + i:start[r] + i + m, h * G:(h + 1) * G].double()
                x = torch.einsum("mgd,ld->mgl", q, k) / math.sqrt(s["D"])
                ago = (seq[r] - n + i + torch.arange(m, device=DEV))[:, None] - torch.arange(seq[r], device=DEV)[None, :]
                hide = ago < 0
                if s["window"]:
                    hide |= (ago >= s["window"]) & (torch.arange(seq[r], device=DEV) >= s["sinks"])
                x.masked_fill_(hide[:, None], -math.inf)
                out[start[r] + i:start[r] + i + m, h * G:(h + 1) * G] = torch.einsum("mgl,ld->mgd", torch.softmax(x, -1), v)
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    q, k = _exact_rotated(s["q"], s["q_norm"], s), _exact_rotated(s["k"], s["k_norm"], s)
    return [q, _exact_held(k), _exact_held(s["v"])] if case["store"] else [q, k]
