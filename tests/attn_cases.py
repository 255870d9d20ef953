"""What the attention tests share beyond attn_ref: which kernels a case runs,
other values or scales in its cache, and a call with its status."""
import ctypes

import numpy as np
import torch

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw

DEV = "cuda"


def workspace(c, window=0, sinks=0):
    a = fw.FwAttnQ4Args(len(c.lens), c.T, c.max_q, c.n_q, c.n_kv, c.D, c.page, c.cache.shape[0], c.max_blocks, window, sinks, 0.1)
    need = ctypes.c_int64()
    assert fw.lib().fw_attn_q4_workspace(ctypes.byref(a), ctypes.byref(need)) == fw.FW_OK
    return need.value


def unpacked_ahead(c, window=0, sinks=0):
    """Whether the call's key tiles are unpacked ahead of the attention: its
    workspace is then two 16-bit tiles and 256 bytes for each 128 positions that
    the block tables can hold, for each key/value head."""
    tiles = len(c.lens) * -(-c.max_blocks * c.page // 128) * c.n_kv
    return workspace(c, window, sinks) == tiles * (2 * 128 * c.D * 2 + 256)


def call(c, window=0, sinks=0, scale=None, q=None, table=None, status=0, **kw):
    """-> the output in float64; the status word has to be `status`."""
    d = c.device()
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = d["block_table"] if table is None else torch.from_numpy(table).to(DEV)
    out = fw.attn_q4(d["q"] if q is None else q.to(DEV), d["cache"], table, d["q_start"], d["seq_lens"], kw.pop("max_q", c.max_q),
                     scale=scale, window=window, sinks=sinks, status=word, **kw)
    torch.cuda.synchronize()
    assert word.item() == status
    return out.double().cpu().numpy()


def check(c, window=0, sinks=0, scale=None, **kw):
    got = call(c, window, sinks, scale, **kw)
    want, tol = c.reference(window, sinks, scale)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:5].tolist())
    return got


def set_values(c, r, x):
    """Request r's values become x [S, n_kv, D], by way of bf16 and the 4-bit blocks."""
    S = c.lens[r][0]
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    codes, d = ref.quantise(x)
    bits = ref.bf16_bits(d)
    for j in range(S):
        for h in range(c.n_kv):
            ref.write_block(c.cache[c.table[r, j // c.page], h], c.page, c.D, j % c.page, "v", codes[j, h], bits[j, h])
    c.v[r] = ref.values(codes, d).reshape(S, c.n_kv, c.D)


def scale_keys(c, powers):
    """The keys of every request times 2^powers[j] at position j (an array as long as the longest, or one number), exactly: their blocks' scales change."""
    powers = np.broadcast_to(powers, (max(s for s, _ in c.lens),))
    for r, (S, _) in enumerate(c.lens):
        p = powers[:S]
        for j in range(S):
            _, at = ref.places(c.page, c.D, "k", j % c.page)
            for h in range(c.n_kv):
                block = c.cache[c.table[r, j // c.page], h]
                bits = block[at].astype(np.uint32) | block[at + 1].astype(np.uint32) << 8
                bits = ref.bf16_bits((bits << 16).astype(np.uint32).view(np.float32).astype(np.float64) * 2.0 ** p[j])
                block[at], block[at + 1] = bits & 0xFF, bits >> 8
        c.k[r] = c.k[r] * 2.0 ** p[:, None, None]
