"""Plain forms, in 64 bits, of the 8-bit blocks, the linear layer over them and
the norms at the residual stream, written from their definitions."""
import numpy as np

BF16 = 2.0 ** -8   # a rounding to bf16 is off by at most this, relative to the value (half a step)
FP32 = 2.0 ** -24


def _table():
    """The values of the e4m3 codes 0 .. 126 (the non-negative numbers, ascending)."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


VALUES = _table()


def encode(x):
    """float64 -> e4m3 codes (uint8): nearest, ties to the even code; beyond 448 the largest; NaN 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.clip(np.searchsorted(VALUES, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - VALUES[lo], VALUES[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = np.where(up, hi, lo).astype(np.uint8)
    c = np.where(np.signbit(x), c | 0x80, c).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), c)


def decode(c):
    c = np.asarray(c, np.uint8)
    v = np.where((c & 127) == 127, np.nan, VALUES[np.minimum(c & 127, 126)])
    return np.where(c >= 128, -v, v)


def quantise(x, rows):
    """[R, K] -> codes uint8 [R, K], scales float32 [ceil(R / rows), ceil(K / 128)], blocks of rows x 128. The rule's own roundings are fp32's."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    nr, nk = -(-R // rows), -(-K // 128)
    codes, scales = np.zeros((R, K), np.uint8), np.zeros((nr, nk), np.float32)
    with np.errstate(all="ignore"):
        for i in range(nr):
            for j in range(nk):
                b = x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
                m = np.float32(np.maximum(np.abs(b).max(), 2.0 ** -96))
                r = np.float32(448) / m
                scales[i, j] = m / np.float32(448)
                codes[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128] = encode(b.astype(np.float32) * r)
    return codes, scales


def values(codes, scales, rows):
    s = np.repeat(np.repeat(scales.astype(np.float64), rows, 0), 128, 1)[:codes.shape[0], :codes.shape[1]]
    return decode(codes) * s


def linear(x_codes, x_scale, w_codes, w_scale):
    """-> [T, N] and how far fp32 sums may be off it. x_scale [T, KB].

    Within a block: at most 128 additions in the tensor core, each off by 2^-23 (should it cut off) of the sum
    of magnitudes; a scale product, its product with the block's sum and the addition over blocks: 2^-24 each."""
    x, w = values(x_codes, x_scale, 1), values(w_codes, w_scale, 128)
    kb = -(-x.shape[1] // 128)
    return x @ w.T, (2 * 128 + 2 + kb) * FP32 * (np.abs(x) @ np.abs(w).T)


def norm_residual(y, residual, norm, post, gate, scale, eps):
    """-> r, h in 64 bits."""
    r = np.asarray(y, np.float64)
    if post is not None:
        r = r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * post
    if gate is not None:
        r = r * gate
    r = r * scale
    big = np.abs(r)
    if residual is not None:
        big = big + np.abs(residual)
        r = r + residual
    h = r if norm is None else r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * norm
    return r, h, big
