"""RMS norm with the residual's addition, in float64 numpy.

    y  = h w / sqrt(mean h^2 + eps)
    dh = rstd (w dy - h rstd^2 mean(w dy h)) + dr,   dw = sum_m dy h rstd

h is the sum as it is stored: the caller rounds x + r to the stream's type.
"""

from __future__ import annotations

import numpy as np


def rstd(h: np.ndarray, eps: float) -> np.ndarray:
    h = np.asarray(h, np.float64)
    return 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(np.float32(eps)))


def fwd(h, w, eps: float) -> np.ndarray:
    return np.asarray(h, np.float64) * rstd(h, eps) * np.asarray(w, np.float64)


def bwd(dy, h, w, eps: float, dr=None):
    """(dh, dw)."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, w))
    rs = rstd(h, eps)
    g = dy * w
    dh = rs * (g - h * rs * rs * (g * h).mean(axis=1, keepdims=True))
    if dr is not None:
        dh = dh + np.asarray(dr, np.float64)
    return dh, (dy * h * rs).sum(axis=0)
