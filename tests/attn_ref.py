"""Plain 64-bit forms of the attention side: the 4-bit block rule, the page
format written byte by byte, the rotation, the plan and the attention with a
bound on what the kernels' roundings may add."""
import math

import numpy as np
import torch

U = 2.0 ** -8  # unit roundoff of bf16: 8 significant bits


def quantise(x):
    """[..., D] (values exact in bf16) -> codes 0..15, scales (float64), by the block rule."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    hi, lo = b.max(-1, keepdims=True), b.min(-1, keepdims=True)
    d = np.where(hi >= -lo, hi, lo) / -8.0
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(d != 0, np.rint(b / d), 0.0) + 8
    return np.clip(c, 0, 15).astype(np.int64).reshape(x.shape), d[..., 0]


def values(codes, scales):
    return (codes.reshape(*scales.shape, 32) - 8) * scales[..., None]


def bf16_bits(x):
    """float64 values exact in bf16 -> their 16 bits."""
    f = np.asarray(x, np.float32).view(np.uint32)
    assert not (f & 0xFFFF).any()
    return (f >> 16).astype(np.uint16)


def page_bytes(page, D):
    return page * D * 9 // 8


def places(page, D, which, at):
    """Where positions `at` (array, places in a page) lie in a (page, head) block: nibble indexes of their D codes, byte indexes of their scales."""
    nb, at = D // 32, np.asarray(at)[..., None]
    d = np.arange(D)
    b, r = d // 32, d % 32
    if which == "k":
        return 2 * (at * (D // 2) + ((r // 8) * nb + b) * 4) + (r % 8) // 2 + 4 * (r % 2), page * D // 2 + 2 * (at * nb + np.arange(nb))
    base = page * D // 2 + page * nb * 2
    return (2 * (base + (at // 2) * D + ((r // 4) * nb + b) * 4) + r % 4 + 4 * (at % 2),
            base + page * D // 2 + 4 * ((at // 2) * nb + np.arange(nb)) + 2 * (at % 2))


def write_block(block, page, D, at, which, codes, scale_bits):
    """Stores one position's D codes and D / 32 scale words (bf16 bits) into a uint8 (page, head) block."""
    nibble, scale_at = places(page, D, which, at)
    shift = 4 * (nibble % 2)
    np.bitwise_and.at(block, nibble // 2, (0xF0 >> shift).astype(np.uint8))
    np.bitwise_or.at(block, nibble // 2, (codes << shift).astype(np.uint8))
    block[scale_at], block[scale_at + 1] = scale_bits & 0xFF, scale_bits >> 8


def rotate(x, norm, eps, cos_sin, positions, interleaved):
    """x [T, heads, D] float64 -> normed and rotated, and the largest magnitude any product of it has."""
    y = x.astype(np.float64)
    if norm is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * norm
    rot = cos_sin.shape[1]
    cs = cos_sin.astype(np.float64)[positions][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + 1 if interleaved else i + rot // 2
    out = y.copy()
    out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
    return out, np.abs(y).max(-1, keepdims=True)


def plan(ctx, new, table, free, page, T_cap, used=0):
    """-> table, q_start, seq_lens, requests, positions, slots, counts as lists."""
    table, start, req, pos, slot, bits = [list(r) for r in table], [0], [], [], [], 0
    lens = []
    for r, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0 or c + n > 1 << 30:
            c = n = 0
            bits |= 8
        if -(-(c + n) // page) > len(table[r]):
            bits |= 2
        for b in range(-(-c // page), -(-(c + n) // page)):
            if b < len(table[r]) and len(req) + b * page - c < T_cap:  # else the token that opens it has no place
                table[r][b] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            e = table[r][p // page] if p // page < len(table[r]) else -1
            req.append(r)
            pos.append(p)
            slot.append(-1 if e < 0 else e * page + p % page)
        start.append(len(req))
        lens.append(c + n)
    bits |= (1 if used > len(free) else 0) | (4 if len(req) > T_cap else 0)
    pad = [-1] * (T_cap - len(req))
    return table, start, lens, (req + pad)[:T_cap], (pos + pad)[:T_cap], (slot + pad)[:T_cap], [len(req), used, bits]


def attention(q, k, v, n_new, scale, window, sinks):
    """One request: q [n, n_q, D], k and v [S, n_kv, D] float64 -> out and an
    elementwise bound. Roundings of relative size U / sqrt(3) (uniform within U)
    on each probability (twice: itself, and times the scale of its block), each
    value and each key's product, taken as independent, at eight standard
    deviations; and the output's own rounding."""
    n, n_q, D = q.shape
    S, n_kv, _ = k.shape
    g = n_q // n_kv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        p = S - n_new + i
        j = np.arange(S)
        see = (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))
        if not see.any():
            continue
        for h in range(n_q):
            kk, vv = k[see, h // g], v[see, h // g]
            s = kk @ q[i, h] * scale
            tau = scale * np.sqrt((kk * kk) @ (q[i, h] * q[i, h])) * U / math.sqrt(3)
            w = np.exp(s - s.max())
            w /= w.sum()
            o = w @ vv
            var = U * U * ((w * w) @ (vv * vv)) + (w * w * tau * tau) @ ((vv - o) ** 2)
            out[i, h] = o
            tol[i, h] = U * np.abs(o) + 8 * np.sqrt(var) + 1e-5 * np.abs(vv).max()
    return out, tol


class Case:
    """A ragged batch over a cache on the device: lens = [(seq_len, new tokens)]."""

    def __init__(self, lens, n_q, n_kv, D, page, seed=0, extra_pages=3, q_gain=1.5, fill=0x7F):
        rng = np.random.default_rng(seed)
        self.lens, self.n_q, self.n_kv, self.D, self.page = lens, n_q, n_kv, D, page
        need = [-(-s // page) for s, _ in lens]
        n_pages = sum(need) + extra_pages
        order = rng.permutation(n_pages)
        self.max_blocks = max(need + [1]) + 1
        table = np.full((len(lens), self.max_blocks), -1, np.int32)
        # what no request owns is garbage: 0xFF.. scales are NaN
        byte = 0xFF if fill is None else fill
        nibbles = np.empty((n_pages, n_kv, page_bytes(page, D), 2), np.uint8)
        nibbles[..., 0], nibbles[..., 1] = byte & 15, byte >> 4
        flat = nibbles.reshape(n_pages, n_kv, -1)
        heads = np.arange(n_kv)[None, :, None]
        self.k, self.v, at = [], [], 0
        for r, (S, _) in enumerate(lens):
            table[r, :need[r]] = order[at:at + need[r]]
            at += need[r]
            kv = []
            for which in "kv":
                x = torch.from_numpy(rng.standard_normal((S, n_kv, D))).to(torch.bfloat16).double().numpy()
                c, d = quantise(x)
                bits = bf16_bits(d)
                j = np.arange(S)
                pages, (nibble, scale_at) = table[r, j // page][:, None, None], places(page, D, which, j % page)
                flat[pages, heads, nibble[:, None]] = c
                for n in range(4):
                    flat[pages, heads, 2 * scale_at[:, None] + n] = bits >> (4 * n) & 15
                kv.append(values(c, d).reshape(x.shape))
            self.k.append(kv[0])
            self.v.append(kv[1])
        starts = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
        self.T, self.max_q = int(starts[-1]), max([n for _, n in lens] + [0])
        self.q = torch.from_numpy(q_gain * rng.standard_normal((self.T, n_q, D))).to(torch.bfloat16)
        self.table, self.starts, self.cache = table, starts, nibbles[..., 0] | nibbles[..., 1] << 4
        self.seq = np.array([s for s, _ in lens], np.int32)

    def device(self, dev="cuda"):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        return dict(q=self.q.to(dev), cache=t(self.cache), block_table=t(self.table), q_start=t(self.starts), seq_lens=t(self.seq))

    def reference(self, window=0, sinks=0, scale=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        q = self.q.double().numpy()
        parts = [attention(q[self.starts[r]:self.starts[r + 1]], self.k[r], self.v[r], n, scale, window, sinks)
                 for r, (_, n) in enumerate(self.lens)]
        return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])
