"""Microscaled (MX) tensors and the RMS norm, from their definitions in fp64.

OCP Microscaling Formats v1.0: elements E2M1 (sign, 2 exponent bits with bias
1, 1 mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6) or E4M3 (codecs.py), 32 of them
sharing one E8M0 scale 2^(b - 127), b = 255 being NaN.  A row's scales take
cols / 32 bytes rounded up to whole 16, the rest zero.
"""
from __future__ import annotations

import numpy as np

from . import codecs

E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EMAX = {"E2M1": 2, "E4M3": 8}
BLOCK = 32


def scale_pitch(cols: int) -> int:
    return -(-(cols // BLOCK) // 16) * 16


def f64_to_e2m1(x: np.ndarray) -> np.ndarray:
    """Nearest e2m1 code, ties to the even code, saturating at 6."""
    m = np.abs(np.asarray(x, dtype=np.float64))
    mid = (E2M1_VALUES[1:] + E2M1_VALUES[:-1]) / 2
    below = np.searchsorted(mid, m, side="left")     # a midpoint itself: the lower code
    tie = (below < 7) & (m == mid[np.minimum(below, 6)]) & (below % 2 == 1)
    code = below + tie                               # an odd lower code: the even one above
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def e2m1_to_f64(code: np.ndarray) -> np.ndarray:
    c = np.asarray(code, dtype=np.uint8)
    v = E2M1_VALUES[c & 7]
    return np.where(c & 8, -v, v)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(b: np.ndarray) -> np.ndarray:
    b = np.asarray(b, dtype=np.uint8)
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def quantize(x: np.ndarray, fmt: str):
    """(codes, scales) of a matrix, as bytes."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - EMAX[fmt], -127)
    e = np.maximum(e, -127)
    v = np.where(bad[..., None], 0.0, np.where(np.isfinite(b), b, 0.0) * np.ldexp(1.0, -e)[..., None]).reshape(rows, cols)
    codes = pack(f64_to_e2m1(v)) if fmt == "E2M1" else codecs.f64_to_e4m3(v)
    scales = np.zeros((rows, scale_pitch(cols)), dtype=np.uint8)
    scales[:, :cols // BLOCK] = np.where(bad, 255, e + 127)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, fmt: str, cols: int) -> np.ndarray:
    v = e2m1_to_f64(unpack(codes)) if fmt == "E2M1" else codecs.e4m3_to_f64(codes)
    s = np.asarray(scales, dtype=np.uint8)[..., :cols // BLOCK].astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(f, BLOCK, axis=-1)


def rms_norm(h: np.ndarray, weight: np.ndarray, eps: float):
    """(y, rstd) of rows."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * np.asarray(weight, dtype=np.float64), rstd


def rms_norm_backward(dy, h, weight, rstd, dh=None):
    """(dx, dweight)."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, weight))
    n = h * np.asarray(rstd, dtype=np.float64)[:, None]
    g = dy * w
    dx = (g - n * (g * n).mean(-1, keepdims=True)) * np.asarray(rstd, dtype=np.float64)[:, None]
    return (dx if dh is None else dx + dh), (dy * n).sum(0)
