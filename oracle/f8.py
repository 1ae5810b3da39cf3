"""F8 tensors (E4M3 elements, a power-of-two scale per block of 128) and the
layer norm, from their definitions in fp64.

A row of `cols` values takes pitch(cols) codes (cols rounded up to 128, the
rest zero) and scale_pitch(cols) E8M0 bytes (the blocks rounded up to 16, the
rest zero): byte b scales its block by 2^(b - 127), b = 255 being NaN.  A
block's scale is the least power of two, from 2^-127 on, that brings its
values within 448; one with an infinity or a NaN has byte 255 and zero codes.
"""
from __future__ import annotations

import numpy as np

from . import codecs

BLOCK = 128


def pitch(cols: int) -> int:
    return -(-cols // BLOCK) * BLOCK


def scale_pitch(cols: int) -> int:
    return -(-(-(-cols // BLOCK)) // 16) * 16


def quantize(x: np.ndarray, square: bool = False):
    """(codes, scales) of a matrix, as bytes; square: 128 x 128 values share a scale."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = np.zeros((rows, pitch(cols)))
    b[:, :cols] = x
    b = b.reshape(rows, -1, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    amax = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    if square:
        for r in range(0, rows, BLOCK):
            bad[r:r + BLOCK] = bad[r:r + BLOCK].any(0)
            amax[r:r + BLOCK] = amax[r:r + BLOCK].max(0)
    m, e = np.frexp(amax)                       # amax = m 2^e; 448 = 0.875 2^9
    X = np.where(amax > 0, np.maximum(e - 9 + (m > 0.875), -127), -127)
    v = np.where(bad[..., None] | ~np.isfinite(b), 0.0, b)
    codes = codecs.f64_to_e4m3((v * np.ldexp(1.0, -X)[..., None]).reshape(rows, -1))
    scales = np.zeros((rows, scale_pitch(cols)), dtype=np.uint8)
    scales[:, :X.shape[1]] = np.where(bad, 255, X + 127)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, cols: int | None = None) -> np.ndarray:
    """The values of an F8 tensor, its padding included unless cols is given."""
    codes = np.asarray(codes, dtype=np.uint8)
    s = np.asarray(scales, dtype=np.uint8)[..., :codes.shape[-1] // BLOCK].astype(np.int64)
    v = codecs.e4m3_to_f64(codes) * np.repeat(np.where(s == 255, np.nan, np.ldexp(1.0, s - 127)), BLOCK, axis=-1)
    return v if cols is None else v[..., :cols]


def layer_norm(h, weight, bias, eps):
    """(y, n, mean, rstd) of rows."""
    h = np.asarray(h, dtype=np.float64)
    mean = h.mean(-1)
    e = h - mean[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((e * e).mean(-1) + eps)
        n = e * rstd[:, None]
        y = n * np.asarray(weight, dtype=np.float64)
        return (y if bias is None else y + np.asarray(bias, dtype=np.float64)), n, mean, rstd


def layer_norm_backward(dy, n, weight, rstd, dh=None):
    """(dx, dweight, dbias) from the normalised rows."""
    dy, n, w = (np.asarray(t, dtype=np.float64) for t in (dy, n, weight))
    g = dy * w
    dx = (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True)) * np.asarray(rstd, dtype=np.float64)[:, None]
    return (dx if dh is None else dx + dh), (dy * n).sum(0), dy.sum(0)
