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


_bf16, _int32, _fp32, _uint8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # not in builds of torch without CUDA

# Small calls last a few microseconds, most of it here: each check is one
# expression, and a message is only made for one that failed.


def _stream(t, stream):
    return stream if stream is not None else _raw_stream(t.get_device())


def _ints(where, name, t):
    if t is not None and not (t.dtype is _int32 and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{where}: {name} must be a contiguous int32 CUDA tensor")


def _heads(where, name, t):
    """Elements between tokens of a bf16 [T, heads, D] tensor whose heads lie side by side."""
    if not (t.dtype is _bf16 and t.is_cuda and t.dim() == 3):
        raise ValueError(f"{where}: {name} must be a bf16 CUDA tensor [T, heads, D]")
    T, heads, D = t.shape
    s = t.stride()
    if T * heads and not (s[2] == 1 and (s[1] == D or heads == 1)):
        raise ValueError(f"{where}: {name}'s heads must be contiguous within a token")
    return s[0] if T > 1 and heads else heads * D


def _cache_page(where, cache, D):
    if not (cache.dtype is _uint8 and cache.is_cuda and cache.dim() == 3 and cache.is_contiguous()):
        raise ValueError(f"{where}: cache must be a contiguous uint8 CUDA tensor [n_pages, n_kv, page * D * 9 / 8]")
    page, rest = divmod(cache.shape[2] * 8, D * 9) if D else (0, 1)
    if rest:
        raise ValueError(f"{where}: cache blocks of {cache.shape[2]} bytes do not hold whole positions of {D} dims")
    return page


def _fail(text):
    raise ValueError(text)


def _keep(stream, *tensors):
    """Tensors made here and used on another stream than the current one stay alive until it is done with them."""
    other = torch.cuda.ExternalStream(stream)
    for t in tensors:
        if t is not None:
            t.record_stream(other)


def kv_cache(n_pages, n_kv, D, page, device="cuda"):
    """An empty 4-bit paged cache: uint8 [n_pages, n_kv, page * D * 9 / 8] (zeros)."""
    return torch.zeros((n_pages, n_kv, page * D * 9 // 8), dtype=torch.uint8, device=device)


def kv_plan(cached_lens, new_lens, block_table, free_pages, page, T_cap, free_used=None, stream=None):
    """The step's plan from the requests' lengths (fw_kv_plan): int32 CUDA tensors
    cached_lens [R], new_lens [R], block_table [R, max_blocks] (fresh entries are
    written), free_pages [n], free_used [1] or None -> KVPlan(q_start [R + 1],
    seq_lens [R], requests, positions, slots [T_cap], counts [3])."""
    for name, t in (("cached_lens", cached_lens), ("new_lens", new_lens), ("block_table", block_table), ("free_pages", free_pages),
                    ("free_used", free_used)):
        _ints("kv_plan", name, t)
    R = cached_lens.shape[0]
    if new_lens.shape != cached_lens.shape or block_table.dim() != 2 or block_table.shape[0] != R:
        _fail("kv_plan: cached_lens [R], new_lens [R] and block_table [R, max_blocks] must agree")
    if T_cap < 1:
        _fail("kv_plan: T_cap must be positive")
    dev = cached_lens.device
    # one buffer for all outputs; its rows are cut where the parts start
    buf = torch.empty(3 * T_cap + 2 * R + 4, dtype=_int32, device=dev)
    if stream is not None:
        _keep(stream, buf)
    at = buf.data_ptr()
    lens = at + 12 * T_cap
    rc = _fw.lib().fw_kv_plan(cached_lens.data_ptr(), new_lens.data_ptr(), R, page, block_table.data_ptr(), block_table.shape[1],
                              free_pages.data_ptr(), free_pages.shape[0], _fw._ptr(free_used), T_cap, lens, lens + 4 * (R + 1),
                              at, at + 4 * T_cap, at + 8 * T_cap, lens + 4 * (2 * R + 1), _stream(buf, stream))
    if rc:
        _fw._check(rc, "fw_kv_plan")
    req, pos, slots, q_start, seq, counts = buf.split((T_cap, T_cap, T_cap, R + 1, R, 3))
    return KVPlan(q_start, seq, req, pos, slots, counts)


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
    if k.shape[0] != T or k.shape[2] != D:
        _fail(f"{w}: q [T, n_q, D] and k [T, n_kv, D] must agree")
    for name, t in (("positions", positions), ("slots", slots), ("status", status)):
        _ints(w, name, t)
    if not (cos_sin.dtype is _fp32 and cos_sin.is_cuda and cos_sin.dim() == 2 and cos_sin.is_contiguous()):
        _fail(f"{w}: cos_sin must be a contiguous fp32 CUDA tensor [n_pos, rot]")
    if positions.shape[0] != T or positions.dim() != 1:
        _fail(f"{w}: positions must be [T]")
    for t in (q_norm, k_norm):
        if t is not None and not (t.dtype is _fp32 and t.is_cuda and t.dim() == 1 and t.shape[0] == D and t.is_contiguous()):
            _fail(f"{w}: norms must be contiguous fp32 CUDA tensors [D]")
    page = n_pages = vs = 0
    if cache is not None:
        page, n_pages = _cache_page(w, cache, D), cache.shape[0]
        if cache.shape[1] != n_kv:
            _fail(f"{w}: cache holds {cache.shape[1]} heads, k has {n_kv}")
        if v is None or v.shape != k.shape:
            _fail(f"{w}: a cache needs v [T, n_kv, D]")
        if slots is None or slots.dim() != 1 or slots.shape[0] != T:
            _fail(f"{w}: a cache needs slots [T]")
        vs = _heads(w, "v", v)
    if q_out is None:
        q_out = torch.empty((T, n_q, D), dtype=_bf16, device=q.device)
        qos = n_q * D
        if stream is not None:
            _keep(stream, q_out)
    else:
        qos = _heads(w, "q_out", q_out)
    kos = 0
    if k_out is not None:
        kos = _heads(w, "k_out", k_out)
    elif cache is None:
        k_out = torch.empty((T, n_kv, D), dtype=_bf16, device=q.device)
        kos = n_kv * D
        if stream is not None:
            _keep(stream, k_out)
    if q_out.shape != q.shape or (k_out is not None and k_out.shape != k.shape):
        _fail(f"{w}: outputs must have their inputs' shapes")
    ptr = _fw._ptr
    args = FwQkNormRopeArgs(T, n_q, n_kv, D, cos_sin.shape[1], 1 if interleaved else 0, eps, cos_sin.shape[0], q.data_ptr(),
                            k.data_ptr(), ptr(v), qs, ks, vs, ptr(q_norm), ptr(k_norm), cos_sin.data_ptr(), positions.data_ptr(),
                            q_out.data_ptr(), ptr(k_out), qos, kos, ptr(cache), ptr(slots), page, n_pages, ptr(status))
    rc = _fw.lib().fw_qk_norm_rope(ctypes.byref(args), _stream(q, stream))
    if rc:
        _fw._check(rc, "fw_qk_norm_rope")
    return q_out, k_out


def kv_export(cache, slots, D, status=None, stream=None):
    """What slots (int32 [T]) of a cache hold (fw_kv_export) -> k, v bf16 [T, n_kv, D]."""
    page = _cache_page("kv_export", cache, D)
    _ints("kv_export", "slots", slots)
    _ints("kv_export", "status", status)
    T, n_kv = slots.shape[0], cache.shape[1]
    k = torch.empty((T, n_kv, D), dtype=_bf16, device=cache.device)
    v = torch.empty((T, n_kv, D), dtype=_bf16, device=cache.device)
    if stream is not None:
        _keep(stream, k, v)
    rc = _fw.lib().fw_kv_export(cache.data_ptr(), cache.shape[0], n_kv, D, page, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(),
                                _fw._ptr(status), _stream(cache, stream))
    if rc:
        _fw._check(rc, "fw_kv_export")
    return k, v


def attn_q4(q, cache, block_table, q_start, seq_lens, max_q, scale=None, window=0, sinks=0, out=None, status=None, stream=None):
    """Causal attention of a step's new tokens over the 4-bit paged cache
    (fw_attn_q4): q bf16 [T, n_q, D], block_table int32 [R, max_blocks], q_start
    int32 [R + 1], seq_lens int32 [R] (new tokens included), max_q the most new
    tokens of a request; scale None: 1 / sqrt(D) -> out bf16 [T, n_q, D]."""
    w = "attn_q4"
    qs = _heads(w, "q", q)
    T, n_q, D = q.shape
    page = _cache_page(w, cache, D)
    for name, t in (("block_table", block_table), ("q_start", q_start), ("seq_lens", seq_lens), ("status", status)):
        _ints(w, name, t)
    R = seq_lens.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] != R or q_start.dim() != 1 or q_start.shape[0] != R + 1:
        _fail(f"{w}: block_table [R, max_blocks], q_start [R + 1] and seq_lens [R] must agree")
    if out is None:
        out = torch.empty((T, n_q, D), dtype=_bf16, device=q.device)
        os = n_q * D
        if stream is not None:
            _keep(stream, out)
    else:
        os = _heads(w, "out", out)
        if out.shape != q.shape:
            _fail(f"{w}: out must have q's shape")
    args = FwAttnQ4Args(R, T, max_q, n_q, cache.shape[1], D, page, cache.shape[0], block_table.shape[1], window, sinks,
                        1.0 / math.sqrt(D) if scale is None else scale, q.data_ptr(), out.data_ptr(), qs, os, cache.data_ptr(),
                        block_table.data_ptr(), q_start.data_ptr(), seq_lens.data_ptr(), _fw._ptr(status))
    L, ref, need, ws = _fw.lib(), ctypes.byref(args), _i64(), None
    rc = L.fw_attn_q4_workspace(ref, ctypes.byref(need))
    if rc:
        _fw._check(rc, "fw_attn_q4_workspace")
    if need.value:
        ws = torch.empty(need.value, dtype=_uint8, device=q.device)
        if stream is not None:
            _keep(stream, ws)
    rc = L.fw_attn_q4(ref, _fw._ptr(ws), need.value, _stream(q, stream))
    if rc:
        _fw._check(rc, "fw_attn_q4")
    return out
