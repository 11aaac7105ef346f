"""The 8-bit integer linear and its row codec, in numpy.

Codec (bit-exact definition, single IEEE fp32 operations): v = x, or
fp32(x * col_scale); scale = fp32(max|v| * fp32(1 / 127)); code = rint(fp32(v / scale)),
half to even, clamped to +-127; 0 where scale is 0; a row that holds a NaN or
an infinity has scale NaN and codes 0.

Linear (float64): Y = (codes_x . codes_w^T) sx sw + sU B^T, and the gradient of
its input through the int8 rows of dY * sw.
"""

from __future__ import annotations

import numpy as np


def quantize(x: np.ndarray, col_scale: np.ndarray | None = None):
    """(codes int8 [M, K], scale float32 [M]) of a float32 matrix."""
    v = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if col_scale is not None:
            v = (v * np.asarray(col_scale, np.float32)[None, :]).astype(np.float32)
        bad = ~np.isfinite(v).all(axis=1)
        c = np.abs(v).max(axis=1)
        s = (c * (np.float32(1) / np.float32(127))).astype(np.float32)
        some = (s > 0) & ~bad
        q = np.zeros(v.shape, np.float32)
        q[some] = np.clip(np.rint((v[some] / s[some, None]).astype(np.float32)), -127, 127)
        s[bad] = np.nan
    return q.astype(np.int8), s


def dequantize_f32(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return (codes.astype(np.float32) * scale[:, None].astype(np.float32)).astype(np.float32)


def _product(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """The exact integer product of int8 matrices (float64 holds it exactly)."""
    return a.astype(np.float64) @ b.astype(np.float64)


def linear_fwd(xq, sx, wq, sw, sU=None, B=None) -> np.ndarray:
    y = _product(xq, wq.T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    return y if sU is None else y + sU @ B.T


def linear_dx(dY_f32, wq, sw, sT=None, A=None) -> np.ndarray:
    gq, sg = quantize(dY_f32, sw)
    d = _product(gq, wq) * sg.astype(np.float64)[:, None]
    return d if sT is None else d + sT @ A
