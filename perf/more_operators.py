"""What a decoder layer needs between its attention and its routed experts: the cases that are measured, and each operator's plain form.

  linear  matrix product in 8-bit floating point (e4m3) with a scale for each block of 128: activations by token and 128 neighbours along K, weights by 128 x 128
  norm    norms after a block and before the next one, fused with the block's gate, the residual scale and the sum; "chain": its result in 8 bits, given to a linear
  route   routing to experts: softmax or sigmoid scores, a bias for balance, groups, top-k, weights renormalised or not
  moe     the routed feed-forward (Q8_0 experts) under such a rule

Definitions:
  linear  a group x of 128: m = max(largest magnitude, 2^-96), scale = m / 448, codes = e4m3(x * (448 / m)), all in fp32; out[t, n] = sum over k of (code * scale)(x) (code * scale)(w)
  norm    r = residual + scale * gate * y / sqrt(mean(y^2) + eps) * post_norm;  h = r / sqrt(mean(r^2) + eps) * norm
  route   z = x Wr^T; s = sigmoid(z) or softmax(z); c = s + bias; a group's score is the sum of its best two c; of the best groups the k experts of largest c; gates = scale * s (over their sum)
  moe     out = sum over the chosen of gate * W_down (SiLU(W_gate x) * W_up x)
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token through a query/key/value projection: latency
        dict(name="linear_token", op="linear", T=1, K=2048, N=5120, out="bf16"),
        # a decode step of a busy server through a large square projection
        dict(name="linear_batch", op="linear", T=64, K=7168, N=7168, out="bf16"),
        # the logits of a decode step, over a large vocabulary
        dict(name="linear_logits", op="linear", T=16, K=2048, N=151936, out="fp32"),
        # a chunk of a prompt, of odd lengths: K ends inside a block, N and T inside a tile
        dict(name="linear_odd", op="linear", T=333, K=4000, N=2051, out="fp32"),
        # a prompt
        dict(name="linear_prompt", op="linear", T=4096, K=7168, N=4096, out="bf16"),
        # one user's next token between two blocks: latency
        dict(name="norm_token", op="norm", T=1, H=2048, residual="bf16", post=False, gate="none", scale=1.0),
        # a prompt through a large model with norms on both sides of a block and a gate for each channel
        dict(name="norm_prompt", op="norm", T=4096, H=7168, residual="bf16", post=True, gate="channel", scale=0.5),
        # a chunk, the residual stream in fp32, a gate for each token
        dict(name="norm_odd", op="norm", T=1001, H=1000, residual="fp32", post=False, gate="token", scale=1.0),
        # the norm before a block with the projection that follows it
        dict(name="chain_prompt", op="chain", T=2048, K=2048, N=5120, residual="bf16", post=False, gate="none", scale=1.0),
        # one user's next token through a router with groups
        dict(name="route_token", op="route", T=1, H=7168, E=256, k=8, score="sigmoid", n_group=8, top_group=4, renorm=True, scale=2.5),
        # a prompt through it
        dict(name="route_prompt", op="route", T=4096, H=7168, E=256, k=8, score="sigmoid", n_group=8, top_group=4, renorm=True, scale=2.5),
        # a decode step through router and experts
        dict(name="moe_batch", op="moe", T=16, H=2048, I=768, E=128, k=8, score="softmax", n_group=1, top_group=1, renorm=False, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rule(rng, E, k):
    n_group = rng.choice([g for g in (1, 4, 8) if E // g >= 2])
    top_group = rng.choice([g for g in range(1, n_group + 1) if g * (E // n_group) >= k])
    return dict(score=rng.choice(["softmax", "sigmoid"]), n_group=n_group, top_group=top_group, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "norm", "norm", "chain", "route", "moe"])
    if op == "linear":
        T, K = _log(rng, 1, 4096), 16 * _log(rng, 16, 448)
        N = _log(rng, 64, 4096) if T > 64 else _log(rng, 64, 100000)
        return dict(op=op, T=T, K=K, N=N, out=rng.choice(["bf16", "bf16", "fp32"]))
    more = dict(residual=rng.choice(["bf16", "bf16", "fp32", "none"]), post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token", "full"]), scale=rng.choice([1.0, 0.5]))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 4096), H=8 * _log(rng, 8, 896), **more)
    if op == "chain":
        return dict(op=op, T=_log(rng, 1, 4096), K=16 * _log(rng, 16, 448), N=_log(rng, 64, 4096), **more)
    E = rng.choice([8, 64, 160, 256])
    k = min(rng.choice([1, 4, 6, 8]), E // 2)
    if op == "route":
        return dict(op=op, T=_log(rng, 1, 4096), H=rng.choice([1024, 2048, 7168]), E=E, k=k, **_rule(rng, E, k))
    E = min(E, 64)
    return dict(op=op, T=_log(rng, 1, 400), H=rng.choice([1024, 2048]), I=64 * rng.randint(2, 12), E=E, k=k, **_rule(rng, E, k))


def work(case):
    op, T = case["op"], case["T"]
    if op in ("route", "moe"):
        H, E, k = case["H"], case["E"], case["k"]
        if op == "route":
            return {"bytes": 4 * E * H + 2 * T * H + 8 * T * k, "flops": 2 * T * E * H}
        touched = E * (1 - (1 - k / E) ** T)  # experts, on average
        return {"bytes": touched * 3 * case["I"] * H * 34 // 32 + 4 * E * H + 4 * T * H + 4 * T * k, "flops": 2 * T * E * H + 6 * T * k * H * case["I"]}
    nbytes = flops = 0
    if op != "linear":
        H, gate = case["K"] if op == "chain" else case["H"], case["gate"]
        nbytes += 2 * T * H + {"bf16": 4, "fp32": 8, "none": 2}[case["residual"]] * T * H + 4 * H * (1 + case["post"])
        nbytes += {"none": 0, "channel": 4 * H, "token": 2 * T, "full": 2 * T * H}[gate] + (2 * T * H if op == "norm" else 0)
        flops += 12 * T * H
    if op != "norm":
        K, N = case["K"], case["N"]
        nbytes += N * K + 4 * -(-N // 128) * -(-K // 128) + (4 if case.get("out") == "fp32" else 2) * T * N + (2 * T * K if op == "linear" else 0)
        flops += 2 * T * N * K
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ blocks of 8 bits, as torch operations
def _padded(x, rows, cols):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _groups(x, rows):
    """fp32 [R, K] -> codes (e4m3, [R, K]) and scales (fp32, [R / rows, K / 128], rounded up) of blocks of rows x 128."""
    b = _padded(x, rows, 128).unflatten(0, (-1, rows)).unflatten(2, (-1, 128))
    m = b.abs().amax((1, 3), keepdim=True).clamp(min=2.0 ** -96)
    top = torch.full_like(m, 448.0)  # (a tensor: by a plain number torch divides with its reciprocal)
    codes = (b * (top / m)).flatten(2).flatten(0, 1)[:x.shape[0], :x.shape[1]].to(torch.float8_e4m3fn)
    return codes.contiguous(), (m / top)[:, 0, :, 0].contiguous()


def _values(codes, scales, rows):
    s = scales.repeat_interleave(rows, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]
    return codes.float() * s


def _q8_0(w):
    """fp32 [..., K] -> Q8_0 blocks, uint8 [..., K / 32 * 34]."""
    b = w.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127.0
    q = torch.where(d > 0, torch.round(b / d), torch.zeros_like(b)).clamp(-127, 127).to(torch.int8)
    return torch.cat((d.half().view(torch.uint8), q.view(torch.uint8)), -1).flatten(-2)


def _q8_0_values(blocks, kind=torch.float32):
    b = blocks.unflatten(-1, (-1, 34))
    return (b[..., :2].contiguous().view(torch.float16).to(kind) * b[..., 2:].contiguous().view(torch.int8).to(kind)).flatten(-2)


# ------------------------------------------------------------------ inputs
def _scores(s, z):
    return torch.sigmoid(z) if s["score"] == "sigmoid" else torch.softmax(z, -1)


def _near_a_tie(s, x):
    """Tokens for which a choice hangs on less than what sums in fp32 differ by: no order of experts is right for them."""
    c = _scores(s, x.double() @ s["router_w"].double().t()) + s["bias"].double()
    g = c.unflatten(1, (s["n_group"], -1)).topk(2, -1).values.sum(-1).sort(1, descending=True)
    kept = torch.zeros_like(g.values).scatter_(1, g.indices[:, :s["top_group"]], 1.0).repeat_interleave(s["E"] // s["n_group"], 1)
    top = torch.where(kept > 0, c, -torch.inf).topk(min(s["k"] + 1, s["E"]), 1).values
    far = 5e-5 * c.abs().amax(1)
    close = (top[:, :-1] - top[:, 1:] < far[:, None]).any(1)
    return close | (g.values[:, :-1] - g.values[:, 1:] < far[:, None])[:, s["top_group"] - 1:s["top_group"]].any(1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    op, T = case["op"], case["T"]
    if op in ("linear", "chain"):
        K, N = case["K"], case["N"]
        s["w"], s["w_scale"] = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(-(-N // 128), -(-K // 128), device=DEV)
        for i in range(0, N, 16384):  # a stretch of rows at a time, to bound what the quantiser holds
            n = min(16384, N - i)
            s["w"][i:i + n], s["w_scale"][i // 128:-(-(i + n) // 128)] = _groups(normal(n, K) * K ** -0.5, 128)
    if op == "linear":
        # activations have channels and tokens that are larger than others
        s["x"] = (normal(T, K) * torch.exp(0.5 * normal(K)) * torch.exp(0.5 * normal(T, 1))).bfloat16()
        s["type"] = torch.float32 if case["out"] == "fp32" else torch.bfloat16
    if op in ("norm", "chain"):
        H = case["K"] if op == "chain" else case["H"]
        s["y"] = normal(T, H).bfloat16()
        s["residual"] = None if case["residual"] == "none" else (3.0 * normal(T, H)).to(torch.float32 if case["residual"] == "fp32" else torch.bfloat16)
        s["norm"], s["post"] = 1.0 + 0.1 * normal(H), 1.0 + 0.1 * normal(H) if case["post"] else None
        gate = case["gate"]
        s["gate"] = {"none": lambda: None, "channel": lambda: 0.3 * normal(H), "token": lambda: torch.sigmoid(normal(T, 1)).bfloat16(),
                     "full": lambda: torch.sigmoid(normal(T, H)).bfloat16()}[gate]()
    if op in ("route", "moe"):
        H, E = case["H"], case["E"]
        s["router_w"], s["bias"] = normal(E, H) * 0.85 * H ** -0.5, 0.02 * normal(E) * (1.0 if case["score"] == "sigmoid" else 1.0 / E)
        s["x"] = normal(T, H).bfloat16()
        for _ in range(60):
            near = _near_a_tie(s, s["x"]).nonzero()[:, 0]
            if not near.numel():
                break
            s["x"][near] = normal(near.numel(), H).bfloat16()
        I = case.get("I", 64)
        if op == "moe":
            s["experts"] = [_q8_0(0.02 * normal(E, r, c)).flatten(1) for r, c in ((I, H), (I, H), (H, I))]
        if own:  # the layer's handle, made once: weights laid out, workspace
            import quantized_sparse_moe_router_gb300 as fw
            experts = s["experts"] if op == "moe" else [torch.zeros(E, I * H // 32 * 34, dtype=torch.uint8, device=DEV)] * 3
            s["layer"] = fw.MoELayer(H, I, E, case["k"], T_max=T, weights=dict(router_w=s["router_w"], w_gate=experts[0], w_up=experts[1], w_down=experts[2]),
                                     routing=dict(score=s["score"], n_group=s["n_group"], top_group=s["top_group"], renorm=s["renorm"], scale=s["scale"], bias=s["bias"]))
    return s


# ------------------------------------------------------------------ plain forms
def _plain_linear(x, s, kind):
    return (_values(*_groups(x.float(), 1), 1) @ _values(s["w"], s["w_scale"], 128).t()).to(kind)


def _unit(x):
    return x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS))


def _plain_norm(s):
    r = s["y"].float()
    if s["post"] is not None:
        r = _unit(r) * s["post"]
    if s["gate"] is not None:
        r = r * s["gate"].float()
    r = r * s["scale"]
    if s["residual"] is not None:
        r = r + s["residual"].float()
    h = (_unit(r) * s["norm"]).to(torch.bfloat16)
    return r.to(torch.bfloat16 if s["residual"] is None else s["residual"].dtype), h


def _plain_route(s):
    score = _scores(s, s["x"].float() @ s["router_w"].t())
    c = score + s["bias"]
    best = c.unflatten(1, (s["n_group"], -1)).sort(-1, descending=True).values[..., :2].sum(-1)
    kept = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_group"]]
    kept = torch.zeros_like(best).scatter_(1, kept, 1.0).repeat_interleave(s["E"] // s["n_group"], 1)
    ids = torch.where(kept > 0, c, -math.inf).sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    gates = score.gather(1, ids)
    if s["renorm"]:
        gates = gates / (gates.sum(1, keepdim=True) + 1e-20)
    return ids.int(), gates * s["scale"]


def _plain_moe(s):
    ids, gates = _plain_route(s)
    H, I, E = s["H"], s["I"], s["E"]
    g, u, d = (_q8_0_values(b.view(E, r, -1)) for b, r in zip(s["experts"], (I, I, H)))
    x = s["x"].float()
    a = x @ g.transpose(1, 2)  # [E, T, I]
    h = a / (1.0 + torch.exp(-a)) * (x @ u.transpose(1, 2))
    h = h * torch.zeros(s["T"], E, device=DEV).scatter_(1, ids.long(), gates).t()[:, :, None]
    return ids, (h.transpose(0, 1).flatten(1) @ d.transpose(1, 2).flatten(0, 1)).bfloat16()


def run(s):
    op = s["op"]
    if not own:
        if op == "linear":
            return [_plain_linear(s["x"], s, s["type"])]
        if op == "norm":
            return list(_plain_norm(s))
        if op == "chain":
            r, h = _plain_norm(s)
            return [r, _plain_linear(h, s, torch.bfloat16)]
        return list(_plain_route(s) if op == "route" else _plain_moe(s))
    import quantized_sparse_moe_router_gb300 as fw
    if op == "linear":
        return [fw.linear_fp8(s["x"], s["w"], s["w_scale"], out_dtype=s["type"])]
    if op in ("norm", "chain"):
        r, h = fw.norm_residual(s["y"], s["residual"], norm=s["norm"], post_norm=s["post"], gate=s["gate"], scale=s["scale"], eps=EPS, fp8=op == "chain")
        return [r, h] if op == "norm" else [r, fw.linear_fp8(h[0], s["w"], s["w_scale"], x_scale=h[1])]
    if op == "route":
        return list(s["layer"].route(s["x"], gates=torch.empty(s["T"], s["k"], device=DEV)))
    return list(s["layer"].forward(s["x"]))


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_e4m3(v):
    """The e4m3 value nearest to each of v, ties to even: three bits after the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2((torch.frexp(v).exponent - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_linear(x, s):
    """x [T, K] in 64 bits, holding bf16 values."""
    out = 0.0
    w, ws = s["w"].float(), s["w_scale"].double()
    for b in range(ws.shape[1]):
        part = slice(128 * b, min(128 * b + 128, x.shape[1]))
        m = x[:, part].abs().amax(1, keepdim=True).clamp(min=2.0 ** -96)
        codes = _exact_e4m3((x[:, part] * (448.0 / m).float().double()).float().double())  # the rule's own roundings to fp32
        rows = ws[:, b].repeat_interleave(128)[:w.shape[0]]
        out = out + torch.mm(codes * (m / 448.0).float().double(), (w[:, part].double() * rows[:, None]).t())
    return out


def _exact_norm(s):
    H = s["y"].shape[1]
    r = s["y"].double()
    if s["post"] is not None:
        r = r * torch.rsqrt(r.square().sum(1, keepdim=True) / H + EPS) * s["post"].double()
    r = r * (s["scale"] if s["gate"] is None else s["scale"] * s["gate"].double())
    if s["residual"] is not None:
        r = s["residual"].double() + r
    return r, r / torch.sqrt(r.square().sum(1, keepdim=True) / H + EPS) * s["norm"].double()


def _exact_route(s):
    z = torch.einsum("th,eh->te", s["x"].double(), s["router_w"].double())
    p = 1 / (1 + torch.exp(-z)) if s["score"] == "sigmoid" else torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    c, size = p + s["bias"].double(), s["E"] // s["n_group"]
    rows_ids, rows_gates = [], []
    p = p.cpu()
    for t, row in enumerate(c.tolist()):
        score = [sum(sorted(row[g * size:(g + 1) * size])[-2:]) for g in range(s["n_group"])]
        groups = sorted(range(s["n_group"]), key=lambda g: (-score[g], g))[:s["top_group"]]
        ids = sorted((e for g in groups for e in range(g * size, (g + 1) * size)), key=lambda e: (-row[e], e))[:s["k"]]
        w = p[t, ids]
        rows_ids.append(ids)
        rows_gates.append(s["scale"] * (w / (w.sum() + 1e-20) if s["renorm"] else w))
    return torch.tensor(rows_ids, dtype=torch.int32, device=DEV), torch.stack(rows_gates).to(DEV)


def _exact_moe(s):
    ids, gates = _exact_route(s)
    x, out = s["x"].double(), torch.zeros(s["T"], s["H"], dtype=torch.float64, device=DEV)
    for e in range(s["E"]):
        t, slot = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            g, u, d = (_q8_0_values(b[e].view(r, -1), torch.float64) for b, r in zip(s["experts"], (s["I"], s["I"], s["H"])))
            a = x[t] @ g.t()
            out[t] += gates[t, slot][:, None] * ((a * torch.sigmoid(a) * (x[t] @ u.t())) @ d.t())
    return ids, out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return [_exact_linear(s["x"].double(), s)]
    if op == "norm":
        return list(_exact_norm(s))
    if op == "chain":
        r, h = _exact_norm(s)
        return [r, _exact_linear(h.to(torch.bfloat16).double(), s)]
    return list(_exact_route(s) if op == "route" else _exact_moe(s))
