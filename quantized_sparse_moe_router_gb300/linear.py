"""Linear layers in 8 bits and the norms at the residual stream on torch
tensors: quantize_fp8, quantize_fp8_weight, linear_fp8 and norm_residual
(include/fwmoe.h describes the operations, the 8-bit blocks and the errors).
Checks of types and shapes, output allocation and marshalling only; every value
is computed in the library."""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

import quantized_sparse_moe_router_gb300 as _fw

from . import attention as _attention
from .attention import _empty, _empty_on, _fail, _i32, _i64, _f32, _not_ints, _raw_stream, _vp


class FwLinearFp8Args(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("T", "K", "N", "out_fp32")] + [("x", _vp), ("x_scale", _vp), ("x_stride", _i64), ("x_scale_stride", _i64), ("w", _vp), ("w_scale", _vp),
                                                                    ("out", _vp), ("out_stride", _i64), ("status", _vp)])


class FwNormResidualArgs(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("T", "H", "residual_fp32", "gate_fp32", "gate_per_token")] + [("eps", _f32), ("scale", _f32)]
                + [(n, _vp) for n in ("y", "residual", "gate")] + [(n, _i64) for n in ("y_stride", "residual_stride", "gate_stride")]
                + [(n, _vp) for n in ("post_norm", "norm", "residual_out", "h")] + [("residual_out_stride", _i64), ("h_stride", _i64)]
                + [("h_codes", _vp), ("h_scale", _vp), ("h_scale_stride", _i64)])


# The argument structs as the C compiler lays them out (a pointer is a whole number;
# 0 for null): packing one takes a fraction of a ctypes structure's time, and small
# calls are bound by what is done here.
_linear_args = struct.Struct("@4i9q").pack
_norm_args = struct.Struct("@5i2f15q").pack

_bf16, _fp32, _e4m3, _uint8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
_byref = ctypes.byref
# An empty tensor of these sizes, strides and type on the current device, quicker than torch.empty;
# a name of torch's own, so one that may be missing or change.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _new(rows, cols, dtype, like, stream):
    """An empty [rows, cols] tensor for a call on `stream` (None: the current one)."""
    global _empty_strided
    if stream is not None:
        return _empty_on(stream, (rows, cols), dtype, like.device)
    if _empty_strided is not None:
        try:
            return _empty_strided((rows, cols), (cols, 1), dtype)
        except TypeError:  # (not the arguments that this torch's takes)
            _empty_strided = None
    return _empty((rows, cols), dtype=dtype, device=like.device)


def _not_sizes(where):
    _fail(f"{where}: sizes must be below 2^31")


def _rows(where, name, t, cols, *types):
    """Elements between rows of a [T, cols] CUDA tensor whose rows are contiguous."""
    if t.dtype not in types or not t.is_cuda or t.dim() != 2 or t.shape[1] != cols:
        _fail(f"{where}: {name} must be a CUDA tensor [T, {cols}] of {' or '.join(str(x) for x in types)}")
    a, b = t.stride()
    if b != 1 and cols != 1 and t.shape[0]:
        _fail(f"{where}: {name}'s rows must be contiguous")
    return a if t.shape[0] > 1 else cols


def _one_device(where, *tensors):
    if _attention._several is not False:
        _attention._one_device(where, *tensors)


def _blocks(n):
    return (n + 127) // 128


def _scales(K, T, like, stream):
    """fp32 [ceil(K / 128), T] with its rows apart as the library wants them, and how far."""
    stride = (T + 3) // 4 * 4 or 4
    return _new((K + 127) // 128, stride, _fp32, like, stream)[:, :T], stride


def _stream_of(t, stream):
    return _raw_stream(t.get_device()) if stream is None else stream


def quantize_fp8(x, stream=None):
    """bf16 [T, K] -> codes float8_e4m3fn [T, K] and scales fp32 [ceil(K / 128), T] (rows a multiple of
    4 apart): blocks of 128 neighbours of a token (fw_fp8_quantize). K a multiple of 16."""
    w = "quantize_fp8"
    if x.dim() != 2:
        _fail(f"{w}: x must be [T, K]")
    T, K = x.shape
    if T > 0x7FFFFFFF or K > 0x7FFFFFFF:  # (ctypes would cut them to 32 bits)
        _not_sizes(w)
    xs = _rows(w, "x", x, K, _bf16)
    _one_device(w, x)
    codes = _new(T, K, _e4m3, x, stream)
    scales, stride = _scales(K, T, x, stream)
    rc = _fw.lib().fw_fp8_quantize(x.data_ptr(), xs, T, K, codes.data_ptr(), scales.data_ptr(), stride, _stream_of(x, stream))
    if rc:
        _fw._check(rc, "fw_fp8_quantize")
    return codes, scales


def quantize_fp8_weight(w, stream=None):
    """bf16 or fp32 [N, K] -> codes float8_e4m3fn [N, K] and scales fp32 [ceil(N / 128), ceil(K / 128)]:
    blocks of 128 x 128 (fw_fp8_quantize_weight). K a multiple of 16."""
    f = "quantize_fp8_weight"
    if not (w.dtype in (_bf16, _fp32) and w.is_cuda and w.dim() == 2 and w.is_contiguous()):
        _fail(f"{f}: w must be a contiguous bf16 or fp32 CUDA tensor [N, K]")
    N, K = w.shape
    if N > 0x7FFFFFFF or K > 0x7FFFFFFF:
        _not_sizes(f)
    _one_device(f, w)
    codes, scales = _new(N, K, _e4m3, w, stream), _new(_blocks(N), _blocks(K), _fp32, w, stream)
    rc = _fw.lib().fw_fp8_quantize_weight(w.data_ptr(), 1 if w.dtype is _fp32 else 0, N, K, codes.data_ptr(), scales.data_ptr(), _stream_of(w, stream))
    if rc:
        _fw._check(rc, "fw_fp8_quantize_weight")
    return codes, scales


def _linear_refuses(x, w, w_scale, x_scale):
    """Says what is wrong with linear_fp8's inputs."""
    f = "linear_fp8"
    if x.dim() != 2 or w.dim() != 2:
        _fail(f"{f}: x must be [T, K] and w [N, K]")
    (T, K), N = x.shape, w.shape[0]
    if not (w.dtype is _e4m3 and w.is_cuda and w.is_contiguous() and w.shape[1] == K):
        _fail(f"{f}: w must be a contiguous float8_e4m3fn CUDA tensor [N, {K}]")
    _rows(f, "x", x, K, _bf16 if x_scale is None else _e4m3)
    if not (w_scale.dtype is _fp32 and w_scale.is_cuda and w_scale.is_contiguous() and w_scale.shape == (_blocks(N), _blocks(K))):
        _fail(f"{f}: w_scale must be a contiguous fp32 CUDA tensor [{_blocks(N)}, {_blocks(K)}]")
    _fail(f"{f}: x_scale must be an fp32 CUDA tensor [{_blocks(K)}, {T}] with contiguous rows")


@functools.lru_cache(maxsize=1024)
def _linear_workspace(T, K):
    """fw_linear_fp8_workspace's answer for bf16 tokens, which does not depend on N."""
    need = _i64()
    _fw._check(_fw.lib().fw_linear_fp8_workspace(_linear_args(T, K, 1, 0, 0, 0, K, 0, 0, 0, 0, 1, 0), _byref(need)), "fw_linear_fp8_workspace")
    return need.value


def linear_fp8(x, w, w_scale, x_scale=None, out=None, out_dtype=None, status=None, stream=None):
    """x W^T in 8 bits (fw_linear_fp8): x bf16 [T, K], or codes [T, K] with x_scale as quantize_fp8 or
    norm_residual(fp8=True) give them; w codes [N, K] with w_scale as quantize_fp8_weight gives them
    -> [T, N], bf16 or (out_dtype, or out's) fp32."""
    sx, sw, codes = x.shape, w.shape, x_scale is not None
    if len(sx) != 2 or len(sw) != 2:
        _linear_refuses(x, w, w_scale, x_scale)
    T, K = sx
    N = sw[0]
    xs, one = x.stride()
    if not (x.dtype is (_e4m3 if codes else _bf16) and w.dtype is _e4m3 and w_scale.dtype is _fp32 and sw[1] == K and (one == 1 or T == 0)
            and w_scale.shape == ((N + 127) // 128, (K + 127) // 128) and w.is_contiguous() and w_scale.is_contiguous() and x.is_cuda and w.is_cuda
            and w_scale.is_cuda):
        _linear_refuses(x, w, w_scale, x_scale)
    if T < 2:
        xs = K
    s_at = ss = 0
    if codes:
        if not (x_scale.dtype is _fp32 and x_scale.is_cuda and x_scale.shape == ((K + 127) // 128, T) and (x_scale.stride(1) == 1 or T < 2)):
            _linear_refuses(x, w, w_scale, x_scale)
        s_at, ss = x_scale.data_ptr(), x_scale.stride(0)
    if status is not None:
        _not_ints("linear_fp8", status=status)
    if _attention._several is not False:
        _attention._one_device("linear_fp8", x, w, w_scale, x_scale, out, status)
    if out is None:
        if out_dtype is None:
            out_dtype = _bf16
        elif out_dtype is not _bf16 and out_dtype is not _fp32:
            _fail("linear_fp8: out_dtype must be torch.bfloat16 or torch.float32")
        out, os = _new(T, N, out_dtype, x, stream), N
    else:
        if out.dim() != 2 or out.shape[0] != T or out_dtype not in (None, out.dtype):
            _fail("linear_fp8: out must be [T, N] of out_dtype")
        os, out_dtype = _rows("linear_fp8", "out", out, N, _bf16, _fp32), out.dtype
    args = _linear_args(T, K, N, 1 if out_dtype is _fp32 else 0, x.data_ptr(), s_at, xs, ss, w.data_ptr(), w_scale.data_ptr(), out.data_ptr(), os,
                        0 if status is None else status.data_ptr())
    L, size, at = _fw._lib or _fw.lib(), 0, None
    if T > 16 and not codes:  # (otherwise none is needed)
        size = _linear_workspace(T, K)
        ws = _new(1, size, _uint8, x, None) if stream is None else _empty_on(stream, (size,), _uint8, x.device, False)
        at = ws.data_ptr()
    rc = L.fw_linear_fp8(args, at, size, _raw_stream(x.get_device()) if stream is None else stream)
    if rc:
        _fw._check(rc, "fw_linear_fp8")
    return out


def _norm_refuses(y, residual, norm, post_norm):
    """Says what is wrong with norm_residual's inputs."""
    f = "norm_residual"
    if y.dim() != 2:
        _fail(f"{f}: y must be [T, H]")
    T, H = y.shape
    _rows(f, "y", y, H, _bf16)
    if residual is not None:
        _rows(f, "residual", residual, H, _bf16, _fp32)
        if residual.shape[0] != T:
            _fail(f"{f}: residual must be [T, H]")
    _fail(f"{f}: norm and post_norm must be contiguous fp32 CUDA tensors [H]")


def norm_residual(y, residual=None, norm=None, post_norm=None, gate=None, scale=1.0, eps=1e-6, fp8=False, residual_out=None, h=None, stream=None):
    """The norms after a block and before the next one, with the sum between them (fw_norm_residual):
        r = residual + scale * gate * y / sqrt(mean(y^2) + eps) * post_norm,   h = r / sqrt(mean(r^2) + eps) * norm
    y bf16 [T, H]; residual bf16 or fp32 [T, H] or None; gate bf16 or fp32, [H], [T, 1] or [T, H], or None;
    norms fp32 [H] or None -> (r in residual's type, h bf16), or with fp8 (r, (codes, scales)) as
    linear_fp8 takes them. residual_out may be residual."""
    f, shape = "norm_residual", y.shape
    if len(shape) != 2 or y.dtype is not _bf16 or not y.is_cuda:
        _norm_refuses(y, residual, norm, post_norm)
    T, H = shape
    ys, one = y.stride()
    wide = rs = r_at = n_at = p_at = g_at = gs = g_fp32 = g_token = h_at = hs = c_at = s_at = ss = 0
    kind = _bf16
    if residual is not None:
        kind = residual.dtype
        rs, r_one = residual.stride() if residual.dim() == 2 else (0, 0)
        if residual.shape != shape or kind is not _bf16 and kind is not _fp32 or r_one != 1 and T or not residual.is_cuda:
            _norm_refuses(y, residual, norm, post_norm)
        r_at, wide = residual.data_ptr(), 1 if kind is _fp32 else 0
    if norm is not None:
        if not (norm.dtype is _fp32 and norm.shape == (H,) and norm.is_contiguous() and norm.is_cuda):
            _norm_refuses(y, residual, norm, post_norm)
        n_at = norm.data_ptr()
    if post_norm is not None:
        if not (post_norm.dtype is _fp32 and post_norm.shape == (H,) and post_norm.is_contiguous() and post_norm.is_cuda):
            _norm_refuses(y, residual, norm, post_norm)
        p_at = post_norm.data_ptr()
    if one != 1 and T:
        _norm_refuses(y, residual, norm, post_norm)
    if T < 2:
        ys = rs = H
    if gate is not None:
        g = gate.shape
        if gate.dtype is not _bf16 and gate.dtype is not _fp32 or not gate.is_cuda or g not in ((H,), (T, 1), shape, (1, H)):
            _fail(f"{f}: gate must be a bf16 or fp32 CUDA tensor [H], [T, 1] or [T, H]")
        g_at, g_fp32 = gate.data_ptr(), 1 if gate.dtype is _fp32 else 0
        if len(g) == 2 and g[1] == 1 and H != 1:
            g_token, gs = 1, gate.stride(0) if T > 1 else 0
        else:
            if gate.stride(-1) != 1:
                _fail(f"{f}: gate's rows must be contiguous")
            gs = gate.stride(0) if len(g) == 2 and g[0] > 1 else 0
    if _attention._several is not False:
        _attention._one_device(f, y, residual, norm, post_norm, gate, residual_out, h)
    if residual_out is None:
        residual_out, ros = _new(T, H, kind, y, stream), H
    else:
        ros = _rows(f, "residual_out", residual_out, H, kind)
        if residual_out.shape[0] != T:
            _fail(f"{f}: residual_out must be [T, H]")
    if fp8:
        if h is not None:
            _fail(f"{f}: h is bf16, fp8 gives codes and scales")
        codes = _new(T, H, _e4m3, y, stream)
        scales, ss = _scales(H, T, y, stream)
        h, c_at, s_at = (codes, scales), codes.data_ptr(), scales.data_ptr()
    elif h is None:
        h, hs = _new(T, H, _bf16, y, stream), H
        h_at = h.data_ptr()
    else:
        hs = _rows(f, "h", h, H, _bf16)
        if h.shape[0] != T:
            _fail(f"{f}: h must be [T, H]")
        h_at = h.data_ptr()
    rc = (_fw._lib or _fw.lib()).fw_norm_residual(
        _norm_args(T, H, wide, g_fp32, g_token, eps, scale, y.data_ptr(), r_at, g_at, ys, rs, gs, p_at, n_at, residual_out.data_ptr(), h_at, ros, hs, c_at, s_at,
                   ss), _raw_stream(y.get_device()) if stream is None else stream)
    if rc:
        _fw._check(rc, "fw_norm_residual")
    return residual_out, h
