"""Linear layers in 8 bits and the norms at the residual stream on torch
tensors: quantize_fp8, quantize_fp8_weight, linear_fp8 and norm_residual
(include/fwmoe.h describes the operations, the 8-bit blocks and the errors).
Checks of types and shapes, output allocation and marshalling only; every value
is computed in the library."""
from __future__ import annotations

import ctypes
import functools

import torch

import quantized_sparse_moe_router_gb300 as _fw

from .attention import _byref, _empty, _empty_on, _fail, _i32, _i64, _f32, _not_ints, _one_device, _raw_stream, _vp


class FwLinearFp8Args(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("T", "K", "N", "out_fp32")] + [("x", _vp), ("x_scale", _vp), ("x_stride", _i64), ("x_scale_stride", _i64), ("w", _vp), ("w_scale", _vp),
                                                                    ("out", _vp), ("out_stride", _i64), ("status", _vp)])


class FwNormResidualArgs(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("T", "H", "residual_fp32", "gate_fp32", "gate_per_token")] + [("eps", _f32), ("scale", _f32)]
                + [(n, _vp) for n in ("y", "residual", "gate")] + [(n, _i64) for n in ("y_stride", "residual_stride", "gate_stride")]
                + [(n, _vp) for n in ("post_norm", "norm", "residual_out", "h")] + [("residual_out_stride", _i64), ("h_stride", _i64)]
                + [("h_codes", _vp), ("h_scale", _vp), ("h_scale_stride", _i64)])


_bf16, _fp32, _e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _rows(where, name, t, cols, *types):
    """Elements between rows of a [T, cols] CUDA tensor whose rows are contiguous."""
    if t.dtype not in types or not t.is_cuda or t.dim() != 2 or t.shape[1] != cols:
        _fail(f"{where}: {name} must be a CUDA tensor [T, {cols}] of {' or '.join(str(x) for x in types)}")
    a, b = t.stride()
    if b != 1 and cols != 1 and t.shape[0]:
        _fail(f"{where}: {name}'s rows must be contiguous")
    return a if t.shape[0] > 1 else cols


def _blocks(n):
    return (n + 127) // 128


def _scales(new, K, T, device):
    """fp32 [ceil(K / 128), T] with its rows apart as the library wants them, and how far."""
    stride = (T + 3) // 4 * 4 or 4
    return new((_blocks(K), stride), dtype=_fp32, device=device)[:, :T], stride


def _stream_of(t, stream):
    return _raw_stream(t.get_device()) if stream is None else stream


def quantize_fp8(x, stream=None):
    """bf16 [T, K] -> codes float8_e4m3fn [T, K] and scales fp32 [ceil(K / 128), T] (rows a multiple of
    4 apart): blocks of 128 neighbours of a token (fw_fp8_quantize). K a multiple of 16."""
    w = "quantize_fp8"
    if x.dim() != 2:
        _fail(f"{w}: x must be [T, K]")
    T, K = x.shape
    xs = _rows(w, "x", x, K, _bf16)
    _one_device(w, x)
    new = _empty if stream is None else functools.partial(_empty_on, stream)
    codes = new((T, K), dtype=_e4m3, device=x.device)
    scales, stride = _scales(new, K, T, x.device)
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
    _one_device(f, w)
    new = _empty if stream is None else functools.partial(_empty_on, stream)
    codes, scales = new((N, K), dtype=_e4m3, device=w.device), new((_blocks(N), _blocks(K)), dtype=_fp32, device=w.device)
    rc = _fw.lib().fw_fp8_quantize_weight(w.data_ptr(), 1 if w.dtype is _fp32 else 0, N, K, codes.data_ptr(), scales.data_ptr(), _stream_of(w, stream))
    if rc:
        _fw._check(rc, "fw_fp8_quantize_weight")
    return codes, scales


def linear_fp8(x, w, w_scale, x_scale=None, out=None, out_dtype=None, status=None, stream=None):
    """x W^T in 8 bits (fw_linear_fp8): x bf16 [T, K], or codes [T, K] with x_scale as quantize_fp8 or
    norm_residual(fp8=True) give them; w codes [N, K] with w_scale as quantize_fp8_weight gives them
    -> [T, N], bf16 or (out_dtype, or out's) fp32."""
    f = "linear_fp8"
    if x.dim() != 2 or w.dim() != 2:
        _fail(f"{f}: x must be [T, K] and w [N, K]")
    T, K = x.shape
    N = w.shape[0]
    if not (w.dtype is _e4m3 and w.is_cuda and w.is_contiguous() and w.shape[1] == K):
        _fail(f"{f}: w must be a contiguous float8_e4m3fn CUDA tensor [N, {K}]")
    xs = _rows(f, "x", x, K, _bf16 if x_scale is None else _e4m3)
    if not (w_scale.dtype is _fp32 and w_scale.is_cuda and w_scale.is_contiguous() and w_scale.shape == (_blocks(N), _blocks(K))):
        _fail(f"{f}: w_scale must be a contiguous fp32 CUDA tensor [{_blocks(N)}, {_blocks(K)}]")
    ss = 0
    if x_scale is not None:
        if not (x_scale.dtype is _fp32 and x_scale.is_cuda and x_scale.shape == (_blocks(K), T) and (x_scale.stride(1) == 1 or T <= 1)):
            _fail(f"{f}: x_scale must be an fp32 CUDA tensor [{_blocks(K)}, {T}] with contiguous rows")
        ss = x_scale.stride(0)
    if status is not None:
        _not_ints(f, status=status)
    _one_device(f, x, w, w_scale, x_scale, out, status)
    dev = x.device
    if out is None:
        if out_dtype not in (None, _bf16, _fp32):
            _fail(f"{f}: out_dtype must be torch.bfloat16 or torch.float32")
        kind, os = out_dtype or _bf16, N
        out = _empty((T, N), dtype=kind, device=dev) if stream is None else _empty_on(stream, (T, N), kind, dev)
    else:
        if out.dim() != 2 or out.shape[0] != T or out_dtype not in (None, out.dtype):
            _fail(f"{f}: out must be [T, N] of out_dtype")
        os = _rows(f, "out", out, N, _bf16, _fp32)
    a = FwLinearFp8Args(T, K, N, 1 if out.dtype is _fp32 else 0, x.data_ptr(), None if x_scale is None else x_scale.data_ptr(), xs, ss, w.data_ptr(),
                        w_scale.data_ptr(), out.data_ptr(), os, None if status is None else status.data_ptr())
    args, L, need = _byref(a), _fw.lib(), _i64()
    rc = L.fw_linear_fp8_workspace(args, _byref(need))
    if rc:
        _fw._check(rc, "fw_linear_fp8_workspace")
    size, at = need.value, None
    if size:
        ws = _empty(size, dtype=torch.uint8, device=dev) if stream is None else _empty_on(stream, (size,), torch.uint8, dev, False)
        at = ws.data_ptr()
    rc = L.fw_linear_fp8(args, at, size, _stream_of(x, stream))
    if rc:
        _fw._check(rc, "fw_linear_fp8")
    return out


def norm_residual(y, residual=None, norm=None, post_norm=None, gate=None, scale=1.0, eps=1e-6, fp8=False, residual_out=None, h=None, stream=None):
    """The norms after a block and before the next one, with the sum between them (fw_norm_residual):
        r = residual + scale * gate * y / sqrt(mean(y^2) + eps) * post_norm,   h = r / sqrt(mean(r^2) + eps) * norm
    y bf16 [T, H]; residual bf16 or fp32 [T, H] or None; gate bf16 or fp32, [H], [T, 1] or [T, H], or None;
    norms fp32 [H] or None -> (r in residual's type, h bf16), or with fp8 (r, (codes, scales)) as
    linear_fp8 takes them. residual_out may be residual."""
    f = "norm_residual"
    if y.dim() != 2:
        _fail(f"{f}: y must be [T, H]")
    T, H = y.shape
    ys = _rows(f, "y", y, H, _bf16)
    kind, rs, r_at = _bf16, 0, None
    if residual is not None:
        kind = residual.dtype
        rs, r_at = _rows(f, "residual", residual, H, _bf16, _fp32), residual.data_ptr()
        if residual.shape[0] != T:
            _fail(f"{f}: residual must be [T, H]")
    for name, t in (("norm", norm), ("post_norm", post_norm)):
        if t is not None and not (t.dtype is _fp32 and t.is_cuda and t.is_contiguous() and t.shape == (H,)):
            _fail(f"{f}: {name} must be a contiguous fp32 CUDA tensor [H]")
    g_at, gs, g_fp32, g_token = None, 0, 0, 0
    if gate is not None:
        if gate.dtype not in (_bf16, _fp32) or not gate.is_cuda or gate.shape not in ((H,), (T, 1), (T, H), (1, H)):
            _fail(f"{f}: gate must be a bf16 or fp32 CUDA tensor [H], [T, 1] or [T, H]")
        g_at, g_fp32 = gate.data_ptr(), 1 if gate.dtype is _fp32 else 0
        if gate.dim() == 2 and gate.shape[1] == 1 and H != 1:
            g_token, gs = 1, gate.stride(0) if T > 1 else 0
        else:
            if gate.stride(-1) != 1:
                _fail(f"{f}: gate's rows must be contiguous")
            gs = gate.stride(0) if gate.dim() == 2 and gate.shape[0] > 1 else 0
    _one_device(f, y, residual, norm, post_norm, gate, residual_out, h)
    new = _empty if stream is None else functools.partial(_empty_on, stream)
    dev = y.device
    if residual_out is None:
        residual_out, ros = new((T, H), dtype=kind, device=dev), H
    else:
        ros = _rows(f, "residual_out", residual_out, H, kind)
        if residual_out.shape[0] != T:
            _fail(f"{f}: residual_out must be [T, H]")
    h_at, hs, c_at, s_at, ss = None, 0, None, None, 0
    if fp8:
        if h is not None:
            _fail(f"{f}: h is bf16, fp8 gives codes and scales")
        scales, ss = _scales(new, H, T, dev)
        h = new((T, H), dtype=_e4m3, device=dev), scales
        c_at, s_at = h[0].data_ptr(), h[1].data_ptr()
    else:
        if h is None:
            h, hs = new((T, H), dtype=_bf16, device=dev), H
        else:
            hs = _rows(f, "h", h, H, _bf16)
            if h.shape[0] != T:
                _fail(f"{f}: h must be [T, H]")
        h_at = h.data_ptr()
    rc = _fw.lib().fw_norm_residual(_byref(FwNormResidualArgs(
        T, H, 1 if kind is _fp32 else 0, g_fp32, g_token, eps, scale, y.data_ptr(), r_at, g_at, ys, rs, gs, None if post_norm is None else post_norm.data_ptr(),
        None if norm is None else norm.data_ptr(), residual_out.data_ptr(), h_at, ros, hs, c_at, s_at, ss)), _stream_of(y, stream))
    if rc:
        _fw._check(rc, "fw_norm_residual")
    return residual_out, h
