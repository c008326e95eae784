"""8-bit operators in 64 bits (oracle side): block-scaled E4M3 / E5M2 quantization, products, the RMS norm.

Formats (OCP 8-bit floating point): E4M3, bias 7, no infinities, S.1111.111 the only NaN, largest value
448; E5M2, bias 15, infinities and NaNs at exponent 31, largest value 57344.  Scales are E8M0 bytes b,
2^(b - 127), one per 128 elements (or 128 x 128 tile): the least exponent E >= -127 with
amax <= Fmax * 2^E; byte 0 for an all-zero block; a block holding a non-finite element has byte 255 and NaN
codes.
"""
from __future__ import annotations

import numpy as np

from .layout import sf_to_mma

BLOCK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_MANTISSA = {"e4m3": 3, "e5m2": 2}
_BIAS = {"e4m3": 7, "e5m2": 15}
NAN_CODE = 0x7F


def decode(codes, fmt: str) -> np.ndarray:
    """Values of 8-bit codes (fp64)."""
    c = np.asarray(codes).astype(np.int64)
    m, bias = _MANTISSA[fmt], _BIAS[fmt]
    e, f = (c & 0x7F) >> m, c & ((1 << m) - 1)
    v = np.where(e == 0, np.ldexp(f.astype(np.float64), 1 - bias - m),
                 np.ldexp(f.astype(np.float64) + (1 << m), e - bias - m))
    if fmt == "e4m3":
        v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(e == 31, np.where(f == 0, np.inf, np.nan), v)
    return np.where(c & 0x80, -v, v)


def encode(v, fmt: str) -> np.ndarray:
    """Codes of values |v| <= Fmax, round to nearest even, sign of zero kept; NaN -> 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    m, bias = _MANTISSA[fmt], _BIAS[fmt]
    a = np.where(np.isnan(v), 0.0, np.abs(v))
    _, ex = np.frexp(a)                                # a = f * 2^ex, f in [0.5, 1)
    e = np.maximum(ex - 1, 1 - bias)                   # exponent of the binade (or of the subnormals)
    q = np.rint(np.ldexp(a, m - e)).astype(np.int64)   # in units of the binade's step; may reach the next binade
    c = (e + bias - 1) * (1 << m) + q                  # a full binade carries into the exponent
    c = np.where(a == 0, 0, c) | (np.signbit(v).astype(np.int64) << 7)
    return np.where(np.isnan(v), NAN_CODE, c).astype(np.uint8)


def scale_exponent(amax, fmt: str) -> np.ndarray:
    f, ex = np.frexp(np.asarray(amax, dtype=np.float64) / FMAX[fmt])     # amax / Fmax = f * 2^ex
    return np.maximum(np.where(f == 0.5, ex - 1, ex), -127)


def _scale_bytes(amax, fmt):
    finite = np.isfinite(amax)
    b = np.where(amax == 0, 0, scale_exponent(np.where(finite, amax, 0.0), fmt) + 127)
    return np.where(finite, b, 255).astype(np.uint8)


def quantize(x, fmt: str = "e4m3", tile: bool = False):
    """x [rows, cols] -> (codes [rows, cols], scale bytes [rows, ceil(cols / 128)]), blocks along the rows."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    g, gr = -(-cols // BLOCK), -(-rows // BLOCK)
    pad = np.zeros((gr * BLOCK, g * BLOCK))
    with np.errstate(invalid="ignore"):
        pad[:rows, :cols] = np.abs(x)
    if tile:
        amax = np.repeat(pad.reshape(gr, BLOCK, g, BLOCK).max(axis=(1, 3)), BLOCK, axis=0)[:rows]
    else:
        amax = pad[:rows].reshape(rows, g, BLOCK).max(axis=2)
    byte = _scale_bytes(amax, fmt)
    each = np.repeat(byte, BLOCK, axis=1)[:, :cols].astype(np.int64)
    with np.errstate(invalid="ignore"):
        v = np.where(each == 255, np.nan, np.ldexp(np.where(each == 255, 0.0, x), 127 - each))
    return encode(v, fmt), byte


def dequantize(codes, byte, fmt: str = "e4m3") -> np.ndarray:
    codes = np.asarray(codes)
    e = np.repeat(np.asarray(byte, dtype=np.int64), BLOCK, axis=1)[:, : codes.shape[1]]
    return np.where(e == 255, np.nan, np.ldexp(decode(codes, fmt), e - 127))


def mma(byte) -> np.ndarray:
    """Scale bytes in the tensor-core layout."""
    return sf_to_mma(byte)


def gemm(a, b):
    """(A . B^T, sum_k |a b|) of operand values."""
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def rmsnorm(h, weight, eps: float):
    """(y, rstd) in 64 bits."""
    h, w = np.asarray(h, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None):
    """(dh, dweight) in 64 bits for y = h * rstd(h) * weight."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, weight))
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    xh, g = h * r, dy * w
    dh = r * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    if dresidual is not None:
        dh = dh + np.asarray(dresidual, dtype=np.float64)
    return dh, (dy * xh).sum(axis=0)
