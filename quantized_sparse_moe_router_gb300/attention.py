"""The attention side of a layer on torch tensors: kv_plan, qk_norm_rope,
kv_export and attn_q4 (include/fwmoe.h describes the operations, the page
format of the 4-bit cache and the errors). Checks of types and shapes, output
allocation and marshalling only; every value is computed in the library."""
from __future__ import annotations

import collections
import ctypes
import functools
import math

import torch

import quantized_sparse_moe_router_gb300 as _fw

KV_POOL_EMPTY, KV_TABLE_FULL, KV_TOKENS_FULL, KV_BAD_LENGTH, KV_BAD_SLOT, KV_BAD_POSITION, KV_TIMEOUT, KV_BAD_QUERIES = 1, 2, 4, 8, 16, 32, 64, 128

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
_byref = ctypes.byref
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # not in builds of torch without CUDA

_current_device = getattr(torch._C, "_cuda_getDevice", None)
_several = None  # more than one device, once it is known

_empty = torch.empty

# Small calls last a few microseconds on the GPU and more here: what is checked
# is checked in few expressions, and a message is only made for what failed.


def _fail(text):
    raise ValueError(text)


def _not_ints(where, **tensors):
    for name, t in tensors.items():
        if t is not None and not (t.dtype is _int32 and t.is_cuda and t.is_contiguous()):
            _fail(f"{where}: {name} must be a contiguous int32 CUDA tensor")


def _not_heads(where, name, t):
    if not (t.dtype is _bf16 and t.is_cuda and t.dim() == 3):
        _fail(f"{where}: {name} must be a bf16 CUDA tensor [T, heads, D]")
    _fail(f"{where}: {name}'s heads must be contiguous within a token")


def _heads(where, name, t, T, heads, D):
    """Elements between tokens of a bf16 [T, heads, D] tensor whose heads lie side by side."""
    a, b, c = t.stride()
    if t.dtype is not _bf16 or not t.is_cuda or ((c != 1 or (b != D and heads != 1)) and T * heads):
        _not_heads(where, name, t)
    return a if T > 1 and heads else heads * D


def _one_device(where, *tensors):
    """The library launches on the current device: all tensors (or None) have to be there."""
    global _several
    if _several is None:
        _several = torch.cuda.device_count() > 1
    if _several:
        now = _current_device()
        for t in tensors:
            if t is not None and t.get_device() != now:
                _fail(f"{where}: a tensor is on cuda:{t.get_device()}, the current device is cuda:{now}")


def _cache_shape(where, cache, D):
    """-> pages, heads, positions a page."""
    if not (cache.dtype is _uint8 and cache.is_cuda and cache.is_contiguous() and cache.dim() == 3):
        _fail(f"{where}: cache must be a contiguous uint8 CUDA tensor [n_pages, n_kv, page * D * 9 / 8]")
    n_pages, n_kv, size = cache.shape
    page, rest = divmod(size * 8, D * 9) if D else (0, 1)
    if rest:
        _fail(f"{where}: cache blocks of {size} bytes do not hold whole positions of {D} dims")
    return n_pages, n_kv, page


def _empty_on(stream, shape, dtype, device, result=True):
    """Memory for a call on another stream than the current one, out of that
    stream's own pool: what the current stream's pool has may still be in use by
    its queued work, which the other does not wait for. A result is also the
    current stream's from here on."""
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        t = _empty(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def kv_cache(n_pages, n_kv, D, page, device="cuda"):
    """An empty 4-bit paged cache: uint8 [n_pages, n_kv, page * D * 9 / 8] (zeros)."""
    return torch.zeros((n_pages, n_kv, page * D * 9 // 8), dtype=torch.uint8, device=device)


def kv_plan(cached_lens, new_lens, block_table, free_pages, page, T_cap, free_used=None, stream=None):
    """The step's plan from the requests' lengths (fw_kv_plan): int32 CUDA tensors
    cached_lens [R], new_lens [R], block_table [R, max_blocks] (fresh entries are
    written), free_pages [n], free_used [1] or None -> KVPlan(q_start [R + 1],
    seq_lens [R], requests, positions, slots [T_cap], counts [3])."""
    R, blocks = block_table.shape
    if not (cached_lens.dtype is new_lens.dtype is block_table.dtype is free_pages.dtype is _int32 and cached_lens.is_cuda
            and new_lens.is_cuda and block_table.is_cuda and free_pages.is_cuda and cached_lens.is_contiguous()
            and new_lens.is_contiguous() and block_table.is_contiguous() and free_pages.is_contiguous()) or free_used is not None:
        _not_ints("kv_plan", cached_lens=cached_lens, new_lens=new_lens, block_table=block_table, free_pages=free_pages,
                  free_used=free_used)
    if cached_lens.shape != (R,) or new_lens.shape != (R,):
        _fail("kv_plan: cached_lens [R], new_lens [R] and block_table [R, max_blocks] must agree")
    if T_cap < 1:
        _fail("kv_plan: T_cap must be positive")
    _one_device("kv_plan", cached_lens, new_lens, block_table, free_pages, free_used)
    # one buffer for all outputs
    size, dev = 3 * T_cap + 2 * R + 4, block_table.device
    if stream is None:
        buf = _empty(size, dtype=_int32, device=dev)
        stream = _raw_stream(buf.get_device())
    else:
        buf = _empty_on(stream, (size,), _int32, dev)
    at = buf.data_ptr()
    lens = at + 12 * T_cap
    rc = _fw.lib().fw_kv_plan(cached_lens.data_ptr(), new_lens.data_ptr(), R, page, block_table.data_ptr(), blocks,
                              free_pages.data_ptr(), free_pages.shape[0], None if free_used is None else free_used.data_ptr(), T_cap,
                              lens, lens + 4 * (R + 1), at, at + 4 * T_cap, at + 8 * T_cap, lens + 4 * (2 * R + 1), stream)
    if rc:
        _fw._check(rc, "fw_kv_plan")
    req, pos, slots, q_start, seq, counts = buf.split_with_sizes((T_cap, T_cap, T_cap, R + 1, R, 3))
    return KVPlan(q_start, seq, req, pos, slots, counts)


def qk_norm_rope(q, k, positions, cos_sin, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, v=None, cache=None,
                 slots=None, q_out=None, k_out=None, status=None, stream=None):
    """Norms and rotation of queries and keys (fw_qk_norm_rope): q [T, n_q, D], k
    [T, n_kv, D] bf16 (views of a fused projection are fine), positions int32 [T],
    cos_sin fp32 [n_pos, rot], norms fp32 [D] or None. With a cache, the keys and
    v are stored into slots in 4 bits and k_out is made only when it is given.
    -> (q_out, k_out or None)."""
    w = "qk_norm_rope"
    if q.dim() != 3 or k.dim() != 3:
        _not_heads(w, "q" if q.dim() != 3 else "k", q if q.dim() != 3 else k)
    T, n_q, D = q.shape
    shape_k = k.shape
    n_kv = shape_k[1]
    if shape_k[0] != T or shape_k[2] != D:
        _fail(f"{w}: q [T, n_q, D] and k [T, n_kv, D] must agree")
    qs, ks = _heads(w, "q", q, T, n_q, D), _heads(w, "k", k, T, n_kv, D)
    if not (positions.dtype is _int32 and positions.is_cuda and positions.is_contiguous()) or status is not None:
        _not_ints(w, positions=positions, status=status)
    if not (cos_sin.dtype is _fp32 and cos_sin.is_cuda and cos_sin.is_contiguous() and cos_sin.dim() == 2):
        _fail(f"{w}: cos_sin must be a contiguous fp32 CUDA tensor [n_pos, rot]")
    if positions.shape != (T,):
        _fail(f"{w}: positions must be [T]")
    n_pos, rot = cos_sin.shape
    q_norm_at = k_norm_at = None
    for t in (q_norm, k_norm):
        if t is not None and not (t.dtype is _fp32 and t.is_cuda and t.is_contiguous() and t.shape == (D,)):
            _fail(f"{w}: norms must be contiguous fp32 CUDA tensors [D]")
    if q_norm is not None:
        q_norm_at = q_norm.data_ptr()
    if k_norm is not None:
        k_norm_at = k_norm.data_ptr()
    _one_device(w, q, k, positions, cos_sin, q_norm, k_norm, v, cache, slots, q_out, k_out, status)
    page = n_pages = vs = 0
    v_at = cache_at = slots_at = None
    if cache is not None:
        n_pages, heads, page = _cache_shape(w, cache, D)
        if heads != n_kv:
            _fail(f"{w}: cache holds {heads} heads, k has {n_kv}")
        if v is None or v.shape != shape_k:
            _fail(f"{w}: a cache needs v [T, n_kv, D]")
        if slots is None or slots.shape != (T,):
            _fail(f"{w}: a cache needs slots [T]")
        _not_ints(w, slots=slots)
        vs = _heads(w, "v", v, T, n_kv, D)
        v_at, cache_at, slots_at = v.data_ptr(), cache.data_ptr(), slots.data_ptr()
    new = _empty if stream is None else functools.partial(_empty_on, stream)
    if q_out is None:
        q_out, qos = new((T, n_q, D), dtype=_bf16, device=q.device), n_q * D
    else:
        if q_out.shape != q.shape:
            _fail(f"{w}: outputs must have their inputs' shapes")
        qos = _heads(w, "q_out", q_out, T, n_q, D)
    kos, k_out_at = n_kv * D, None
    if k_out is None:
        if cache is None:
            k_out = new((T, n_kv, D), dtype=_bf16, device=q.device)
            k_out_at = k_out.data_ptr()
    else:
        if k_out.shape != shape_k:
            _fail(f"{w}: outputs must have their inputs' shapes")
        kos, k_out_at = _heads(w, "k_out", k_out, T, n_kv, D), k_out.data_ptr()
    if stream is None:
        stream = _raw_stream(q.get_device())
    args = FwQkNormRopeArgs(T, n_q, n_kv, D, rot, 1 if interleaved else 0, eps, n_pos, q.data_ptr(), k.data_ptr(), v_at, qs, ks, vs,
                            q_norm_at, k_norm_at, cos_sin.data_ptr(), positions.data_ptr(), q_out.data_ptr(), k_out_at, qos, kos,
                            cache_at, slots_at, page, n_pages, None if status is None else status.data_ptr())
    rc = _fw.lib().fw_qk_norm_rope(_byref(args), stream)
    if rc:
        _fw._check(rc, "fw_qk_norm_rope")
    return q_out, k_out


def kv_export(cache, slots, D, status=None, stream=None):
    """What slots (int32 [T]) of a cache hold (fw_kv_export) -> k, v bf16 [T, n_kv, D]."""
    n_pages, n_kv, page = _cache_shape("kv_export", cache, D)
    _not_ints("kv_export", slots=slots, status=status)
    _one_device("kv_export", cache, slots, status)
    T = slots.shape[0]
    if stream is None:
        kv = _empty((2, T, n_kv, D), dtype=_bf16, device=cache.device)
        stream = _raw_stream(kv.get_device())
    else:
        kv = _empty_on(stream, (2, T, n_kv, D), _bf16, cache.device)
    at = kv.data_ptr()
    rc = _fw.lib().fw_kv_export(cache.data_ptr(), n_pages, n_kv, D, page, slots.data_ptr(), T, at, at + 2 * T * n_kv * D,
                                None if status is None else status.data_ptr(), stream)
    if rc:
        _fw._check(rc, "fw_kv_export")
    return kv.unbind(0)


def attn_q4(q, cache, block_table, q_start, seq_lens, max_q, scale=None, window=0, sinks=0, out=None, status=None, stream=None):
    """Causal attention of a step's new tokens over the 4-bit paged cache
    (fw_attn_q4): q bf16 [T, n_q, D], block_table int32 [R, max_blocks], q_start
    int32 [R + 1], seq_lens int32 [R] (new tokens included), max_q the most new
    tokens of a request; scale None: 1 / sqrt(D) -> out bf16 [T, n_q, D]."""
    w = "attn_q4"
    if q.dim() != 3:
        _not_heads(w, "q", q)
    T, n_q, D = q.shape
    qs = _heads(w, "q", q, T, n_q, D)
    n_pages, n_kv, page = _cache_shape(w, cache, D)
    if not (block_table.dtype is q_start.dtype is seq_lens.dtype is _int32 and block_table.is_cuda and q_start.is_cuda
            and seq_lens.is_cuda and block_table.is_contiguous() and q_start.is_contiguous()
            and seq_lens.is_contiguous()) or status is not None:
        _not_ints(w, block_table=block_table, q_start=q_start, seq_lens=seq_lens, status=status)
    R, blocks = block_table.shape
    if seq_lens.shape != (R,) or q_start.shape != (R + 1,):
        _fail(f"{w}: block_table [R, max_blocks], q_start [R + 1] and seq_lens [R] must agree")
    _one_device(w, q, cache, block_table, q_start, seq_lens, out, status)
    dev = q.device
    if out is None:
        out = _empty((T, n_q, D), dtype=_bf16, device=dev) if stream is None else _empty_on(stream, (T, n_q, D), _bf16, dev)
        os = n_q * D
    else:
        if out.shape != q.shape:
            _fail(f"{w}: out must have q's shape")
        os = _heads(w, "out", out, T, n_q, D)
    args = _byref(FwAttnQ4Args(R, T, max_q, n_q, n_kv, D, page, n_pages, blocks, window, sinks,
                               1.0 / math.sqrt(D) if scale is None else scale, q.data_ptr(), out.data_ptr(), qs, os,
                               cache.data_ptr(), block_table.data_ptr(), q_start.data_ptr(), seq_lens.data_ptr(),
                               None if status is None else status.data_ptr()))
    L, need = _fw.lib(), _i64()
    rc = L.fw_attn_q4_workspace(args, _byref(need))
    if rc:
        _fw._check(rc, "fw_attn_q4_workspace")
    size, at = need.value, None
    if size:
        ws = _empty(size, dtype=_uint8, device=dev) if stream is None else _empty_on(stream, (size,), _uint8, dev, False)
        at = ws.data_ptr()
    if stream is None:
        stream = _raw_stream(q.get_device())
    rc = L.fw_attn_q4(args, at, size, stream)
    if rc:
        _fw._check(rc, "fw_attn_q4")
    return out
