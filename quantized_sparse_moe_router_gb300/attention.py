"""The attention side of a layer on torch tensors: kv_plan, qk_norm_rope,
kv_export and attn_q4 (include/fwmoe.h describes the operations, the page
format of the 4-bit cache and the errors). Checks of types and shapes, output
allocation and marshalling only; every value is computed in the library."""
from __future__ import annotations

import collections
import ctypes
import math

import torch

import quantized_sparse_moe_router_gb300 as _fw

KV_POOL_EMPTY, KV_TABLE_FULL, KV_TOKENS_FULL, KV_BAD_LENGTH, KV_BAD_SLOT, KV_BAD_POSITION = 1, 2, 4, 8, 16, 32

KVPlan = collections.namedtuple("KVPlan", "q_start seq_lens requests positions slots counts")

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class FwQkNormRopeArgs(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("T", "n_q", "n_kv", "D", "rot", "interleaved")] + [("eps", _f32), ("n_pos", _i32)]
                + [(n, _vp) for n in ("q", "k", "v")] + [(n, _i64) for n in ("q_stride", "k_stride", "v_stride")]
                + [(n, _vp) for n in ("q_norm", "k_norm", "cos_sin", "positions", "q_out", "k_out")]
                + [("q_out_stride", _i64), ("k_out_stride", _i64), ("cache", _vp), ("slots", _vp), ("page", _i32),
                   ("n_pages", _i32), ("status", _vp)])


class FwAttnQ4Args(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("R", "T", "max_q", "n_q", "n_kv", "D", "page", "n_pages", "max_blocks", "window",
                                     "sinks")] + [("scale", _f32), ("q", _vp), ("out", _vp), ("q_stride", _i64),
                                                  ("out_stride", _i64)]
                + [(n, _vp) for n in ("cache", "block_table", "q_start", "seq_lens", "status")])


def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _int32(where, **tensors):
    for name, t in tensors.items():
        if t is not None:
            _need(t.is_cuda and t.dtype == torch.int32 and t.is_contiguous(), f"{where}: {name} must be a contiguous int32 CUDA tensor")


def _heads(where, name, t):
    """A bf16 [T, heads, D] tensor whose heads lie side by side; tokens may be any distance apart."""
    _need(t.is_cuda and t.dtype == torch.bfloat16 and t.dim() == 3, f"{where}: {name} must be a bf16 CUDA tensor [T, heads, D]")
    s = t.stride()
    _need(t.numel() == 0 or (s[2] == 1 and (s[1] == t.shape[2] or t.shape[1] == 1)),
          f"{where}: {name}'s heads must be contiguous within a token")
    return s[0] if t.shape[0] > 1 and t.numel() else t.shape[1] * t.shape[2]


def _cache_page(where, cache, D):
    _need(cache.is_cuda and cache.dtype == torch.uint8 and cache.dim() == 3 and cache.is_contiguous(),
          f"{where}: cache must be a contiguous uint8 CUDA tensor [n_pages, n_kv, page * D * 9 / 8]")
    page, rest = divmod(cache.shape[2] * 8, D * 9)
    _need(rest == 0, f"{where}: cache blocks of {cache.shape[2]} bytes do not hold whole positions of {D} dims")
    return page


def _keep(stream, *tensors):
    """Tensors made here and used on another stream than the current one stay alive until it is done with them."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(torch.cuda.ExternalStream(stream))


def kv_cache(n_pages, n_kv, D, page, device="cuda"):
    """An empty 4-bit paged cache: uint8 [n_pages, n_kv, page * D * 9 / 8] (zeros)."""
    return torch.zeros((n_pages, n_kv, page * D * 9 // 8), dtype=torch.uint8, device=device)


def kv_plan(cached_lens, new_lens, block_table, free_pages, page, T_cap, free_used=None, stream=None):
    """The step's plan from the requests' lengths (fw_kv_plan): int32 CUDA tensors
    cached_lens [R], new_lens [R], block_table [R, max_blocks] (fresh entries are
    written), free_pages [n], free_used [1] or None -> KVPlan(q_start [R + 1],
    seq_lens [R], requests, positions, slots [T_cap], counts [3])."""
    _int32("kv_plan", cached_lens=cached_lens, new_lens=new_lens, block_table=block_table, free_pages=free_pages, free_used=free_used)
    R = cached_lens.shape[0]
    _need(new_lens.shape == (R,) and block_table.dim() == 2 and block_table.shape[0] == R,
          "kv_plan: cached_lens [R], new_lens [R] and block_table [R, max_blocks] must agree")
    _need(T_cap >= 1, "kv_plan: T_cap must be positive")
    lens = torch.empty(2 * R + 4, dtype=torch.int32, device=cached_lens.device)
    toks = torch.empty((3, T_cap), dtype=torch.int32, device=cached_lens.device)
    _keep(stream, lens, toks)
    at, row = lens.data_ptr(), toks.data_ptr()
    _fw._check(_fw.lib().fw_kv_plan(cached_lens.data_ptr(), new_lens.data_ptr(), R, page, block_table.data_ptr(),
                                    block_table.shape[1], free_pages.data_ptr(), free_pages.shape[0],
                                    _fw._ptr(free_used), T_cap, at, at + 4 * (R + 1), row, row + 4 * T_cap, row + 8 * T_cap,
                                    at + 4 * (2 * R + 1), _fw._stream(stream)), "fw_kv_plan")
    return KVPlan(lens[:R + 1], lens[R + 1:2 * R + 1], toks[0], toks[1], toks[2], lens[2 * R + 1:])


def qk_norm_rope(q, k, positions, cos_sin, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, v=None, cache=None,
                 slots=None, q_out=None, k_out=None, status=None, stream=None):
    """Norms and rotation of queries and keys (fw_qk_norm_rope): q [T, n_q, D], k
    [T, n_kv, D] bf16 (views of a fused projection are fine), positions int32 [T],
    cos_sin fp32 [n_pos, rot], norms fp32 [D] or None. With a cache, the keys and
    v are stored into slots in 4 bits and k_out is made only when it is given.
    -> (q_out, k_out or None)."""
    w = "qk_norm_rope"
    qs, ks = _heads(w, "q", q), _heads(w, "k", k)
    T, n_q, D = q.shape
    n_kv = k.shape[1]
    _need(k.shape == (T, n_kv, D), f"{w}: q [T, n_q, D] and k [T, n_kv, D] must agree")
    _int32(w, positions=positions, slots=slots, status=status)
    _need(cos_sin.is_cuda and cos_sin.dtype == torch.float32 and cos_sin.dim() == 2 and cos_sin.is_contiguous(),
          f"{w}: cos_sin must be a contiguous fp32 CUDA tensor [n_pos, rot]")
    _need(positions.shape == (T,), f"{w}: positions must be [T]")
    for t in (q_norm, k_norm):
        _need(t is None or (t.is_cuda and t.dtype == torch.float32 and t.shape == (D,) and t.is_contiguous()),
              f"{w}: norms must be contiguous fp32 CUDA tensors [D]")
    page = n_pages = vs = 0
    if cache is not None:
        page, n_pages = _cache_page(w, cache, D), cache.shape[0]
        _need(cache.shape[1] == n_kv, f"{w}: cache holds {cache.shape[1]} heads, k has {n_kv}")
        _need(v is not None and v.shape == k.shape, f"{w}: a cache needs v [T, n_kv, D]")
        _need(slots is not None and slots.shape == (T,), f"{w}: a cache needs slots [T]")
        vs = _heads(w, "v", v)
    if q_out is None:
        q_out = torch.empty((T, n_q, D), dtype=torch.bfloat16, device=q.device)
        _keep(stream, q_out)
    if k_out is None and cache is None:
        k_out = torch.empty((T, n_kv, D), dtype=torch.bfloat16, device=q.device)
        _keep(stream, k_out)
    _need(q_out.shape == q.shape and (k_out is None or k_out.shape == k.shape), f"{w}: outputs must have their inputs' shapes")
    args = FwQkNormRopeArgs(T, n_q, n_kv, D, cos_sin.shape[1], 1 if interleaved else 0, eps, cos_sin.shape[0], q.data_ptr(),
                            k.data_ptr(), _fw._ptr(v), qs, ks, vs, _fw._ptr(q_norm), _fw._ptr(k_norm), cos_sin.data_ptr(),
                            positions.data_ptr(), q_out.data_ptr(), _fw._ptr(k_out), _heads(w, "q_out", q_out),
                            0 if k_out is None else _heads(w, "k_out", k_out), _fw._ptr(cache), _fw._ptr(slots), page, n_pages,
                            _fw._ptr(status))
    _fw._check(_fw.lib().fw_qk_norm_rope(ctypes.byref(args), _fw._stream(stream)), "fw_qk_norm_rope")
    return q_out, k_out


def kv_export(cache, slots, D, status=None, stream=None):
    """What slots (int32 [T]) of a cache hold (fw_kv_export) -> k, v bf16 [T, n_kv, D]."""
    page = _cache_page("kv_export", cache, D)
    _int32("kv_export", slots=slots, status=status)
    T, n_kv = slots.shape[0], cache.shape[1]
    kv = torch.empty((2, T, n_kv, D), dtype=torch.bfloat16, device=cache.device)
    _keep(stream, kv)
    at = kv.data_ptr()
    _fw._check(_fw.lib().fw_kv_export(cache.data_ptr(), cache.shape[0], n_kv, D, page, slots.data_ptr(), T, at,
                                      at + 2 * T * n_kv * D, _fw._ptr(status), _fw._stream(stream)), "fw_kv_export")
    return kv[0], kv[1]


def attn_q4(q, cache, block_table, q_start, seq_lens, max_q, scale=None, window=0, sinks=0, out=None, status=None, stream=None):
    """Causal attention of a step's new tokens over the 4-bit paged cache
    (fw_attn_q4): q bf16 [T, n_q, D], block_table int32 [R, max_blocks], q_start
    int32 [R + 1], seq_lens int32 [R] (new tokens included), max_q the most new
    tokens of a request; scale None: 1 / sqrt(D) -> out bf16 [T, n_q, D]."""
    w = "attn_q4"
    qs = _heads(w, "q", q)
    T, n_q, D = q.shape
    page = _cache_page(w, cache, D)
    _int32(w, block_table=block_table, q_start=q_start, seq_lens=seq_lens, status=status)
    R = seq_lens.shape[0]
    _need(block_table.dim() == 2 and block_table.shape[0] == R and q_start.shape == (R + 1,),
          f"{w}: block_table [R, max_blocks], q_start [R + 1] and seq_lens [R] must agree")
    if out is None:
        out = torch.empty((T, n_q, D), dtype=torch.bfloat16, device=q.device)
        _keep(stream, out)
    _need(out.shape == q.shape, f"{w}: out must have q's shape")
    args = FwAttnQ4Args(R, T, max_q, n_q, cache.shape[1], D, page, cache.shape[0], block_table.shape[1], window, sinks,
                        1.0 / math.sqrt(D) if scale is None else scale, q.data_ptr(), out.data_ptr(), qs, _heads(w, "out", out),
                        cache.data_ptr(), block_table.data_ptr(), q_start.data_ptr(), seq_lens.data_ptr(), _fw._ptr(status))
    L, ref, need = _fw.lib(), ctypes.byref(args), _i64()
    _fw._check(L.fw_attn_q4_workspace(ref, ctypes.byref(need)), "fw_attn_q4_workspace")
    ws = torch.empty(need.value, dtype=torch.uint8, device=q.device) if need.value else None
    _keep(stream, ws)
    _fw._check(L.fw_attn_q4(ref, _fw._ptr(ws), need.value, _fw._stream(stream)), "fw_attn_q4")
    return out
