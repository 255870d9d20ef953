"""One decoder layer served from end to end: attention over the 4-bit paged
cache, then the routed experts.

    python examples/decoder_layer.py

Three steps of four requests -- their prompts, single tokens replayed as a CUDA
graph, and drafted tokens -- each through

    kv_plan         which pages, slots and positions the step's tokens take
    x W_qkv         (a library matrix product; so is W_o)
    qk_norm_rope    norms and rotation of queries and keys, keys and values
                    into the cache
    attn_q4         attention over the cache
    MoELayer        the routed feed-forward

and at the end a second, empty cache that gets every request whole: both ways
agree up to the roundings of bf16.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_sparse_moe_router_gb300 as fw  # noqa: E402


def rope_table(n_pos, rot, base=10000.0, device="cuda"):
    """fp32 [n_pos, rot]: cosines of the rot / 2 frequencies, then sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


class DecoderLayer:
    """Weights of one layer (random here). window and sinks as in attn_q4."""

    def __init__(self, H=512, n_q=8, n_kv=2, D=64, I=256, E=8, k=2, n_pos=4096, T_max=2048, window=0, sinks=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, sd=1.0: sd * torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.n_q, self.n_kv, self.D, self.window, self.sinks = n_q, n_kv, D, window, sinks
        self.w_qkv = rand(H, (n_q + 2 * n_kv) * D, sd=H ** -0.5).bfloat16()
        self.w_o = rand(n_q * D, H, sd=(n_q * D) ** -0.5).bfloat16()
        self.q_norm, self.k_norm = 1 + rand(D, sd=0.1), 1 + rand(D, sd=0.1)
        self.norm1, self.norm2 = (1 + rand(H, sd=0.1)).bfloat16(), (1 + rand(H, sd=0.1)).bfloat16()
        self.cos_sin = rope_table(n_pos, D)
        q8 = lambda r, c: torch.stack([fw.quantize_q8_0(rand(r, c, sd=c ** -0.5)) for _ in range(E)])  # noqa: E731
        self.moe = fw.MoELayer(H, I, E, k, T_max=T_max,
                               weights=dict(router_w=rand(E, H, sd=H ** -0.5), w_gate=q8(I, H), w_up=q8(I, H), w_down=q8(H, I)))

    def project(self, x):
        """-> q, k, v [T, heads, D]: views of one product, used as they are."""
        h = torch.nn.functional.rms_norm(x, (x.shape[1],), self.norm1, 1e-6)
        y = (h @ self.w_qkv).view(x.shape[0], -1, self.D)
        return y.split((self.n_q, self.n_kv, self.n_kv), 1)

    def attend(self, x, plan, cache, block_table, max_q, status=None):
        """x [T, H] of the plan's tokens -> attention's rows [T, n_q, D]; their keys and values are in the cache from then on."""
        q, k, v = self.project(x)
        T = x.shape[0]
        q, _ = fw.qk_norm_rope(q, k, plan.positions[:T], self.cos_sin, self.q_norm, self.k_norm, v=v, cache=cache,
                               slots=plan.slots[:T], status=status)
        return fw.attn_q4(q, cache, block_table, plan.q_start, plan.seq_lens, max_q, window=self.window, sinks=self.sinks, status=status)

    def forward(self, x, plan, cache, block_table, max_q, status=None):
        o = self.attend(x, plan, cache, block_table, max_q, status)
        x = x + o.view(x.shape[0], -1) @ self.w_o
        h = torch.nn.functional.rms_norm(x, (x.shape[1],), self.norm2, 1e-6)
        return x + self.moe.forward(h)[1]


class Requests:
    """R requests' caches: lengths, block tables and the pool of pages, all on the device."""

    def __init__(self, R, layer, page=32, n_pages=256, max_blocks=64, seed=0):
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.page, self.layer = page, layer
        self.cache = fw.kv_cache(n_pages, layer.n_kv, layer.D, page)
        self.lens, self.block_table = ints(R), ints(R, max_blocks)
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))
        self.free_pages, self.used, self.status = order.int().cuda(), ints(1), ints(1)

    def step(self, x, new_lens, max_q):
        """x [T, H]: the requests' new tokens one after the other, new_lens int32 [R]; no host synchronisation."""
        plan = fw.kv_plan(self.lens, new_lens, self.block_table, self.free_pages, self.page, x.shape[0], free_used=self.used)
        y = self.layer.forward(x, plan, self.cache, self.block_table, max_q, self.status)
        self.lens.copy_(plan.seq_lens)
        self.used.copy_(plan.counts[1:2])
        self.status.bitwise_or_(plan.counts[2:3])
        return y


def run(layer, H=512, prompts=(37, 200, 5, 130), singles=6, drafts=(3, 1, 4, 2), seed=1):
    """The three kinds of step -> outputs per request, cached piece by piece and given whole."""
    R = len(prompts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    xs = [torch.randn(p + singles + d, H, generator=g, device="cuda").bfloat16() for p, d in zip(prompts, drafts)]
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = [[] for _ in range(R)]

    def keep(y, lens):
        for o, part in zip(outs, y.split(list(lens))):
            o.append(part.clone())

    cached = Requests(R, layer)
    keep(cached.step(torch.cat([x[:p] for x, p in zip(xs, prompts)]), ints(prompts), max(prompts)), prompts)

    # single tokens: one graph, replayed
    token, ones = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), ints([1] * R)
    graph = torch.cuda.CUDAGraph()
    state = [t.clone() for t in (cached.lens, cached.used, cached.block_table, cached.cache)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (a first run outside of the capture, on tokens that are taken back)
        token.zero_()
        cached.step(token, ones, 1)
        for t, s in zip((cached.lens, cached.used, cached.block_table, cached.cache), state):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        y = cached.step(token, ones, 1)
    for i in range(singles):
        token.copy_(torch.stack([x[p + i] for x, p in zip(xs, prompts)]))
        graph.replay()
        keep(y, [1] * R)

    keep(cached.step(torch.cat([x[p + singles:] for x, p in zip(xs, prompts)]), ints(drafts), max(drafts)), drafts)

    whole = Requests(R, layer, seed=7)
    lens = [x.shape[0] for x in xs]
    at_once = whole.step(torch.cat(xs), ints(lens), max(lens)).split(lens)
    torch.cuda.synchronize()
    for r in (cached, whole):
        if r.status.item():
            raise RuntimeError(f"the step reported {r.status.item():#x} (KV_* bits)")
    layer.moe.status()
    return [torch.cat(o) for o in outs], list(at_once), cached


def main():
    fw.build()
    layer = DecoderLayer()
    pieces, whole, cached = run(layer)
    for r, (a, b) in enumerate(zip(pieces, whole)):
        diff = (a.float() - b.float()).abs()
        print(f"request {r}: {a.shape[0]} tokens, piece by piece against whole: mean {diff.mean():.2e}, max {diff.max():.2e} "
              f"of values up to {b.abs().max():.1f}")
    pages, n_kv, size = cached.cache.shape
    print(f"pages in use: {cached.used.item()} of {pages}, {n_kv * size} bytes each ({cached.page} positions, "
          f"{8 * size / (2 * cached.page * layer.D):.1f} bits a value)")


if __name__ == "__main__":
    main()
