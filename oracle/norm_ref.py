"""Root-mean-square norm with the residual's addition, and its gradients, in
float64.  Test infrastructure only (see the package header).

The pages give the layer's input no norm; the reading taken is the pre-norm
residual block: s = x + res, y = s / sqrt(mean_c s^2 + eps) * w.
"""

from __future__ import annotations

import numpy as np


def forward(x, w, eps, res=None):
    """(y, s, rstd) of rows x [T,d]."""
    s = np.asarray(x, np.float64)
    if res is not None:
        s = s + np.asarray(res, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s * rstd[:, None] * np.asarray(w, np.float64), s, rstd


def backward(dy, s, w, rstd, ds=None):
    """(dx, dw) given dy; ds is the gradient that reaches s itself.

    With rstd a function of s: d rstd / d s_c = -rstd^3 s_c / d, hence
    dx = rstd (g - xh mean(g xh)) with g = dy w and xh = s rstd.
    """
    dy, s, w = (np.asarray(a, np.float64) for a in (dy, s, w))
    rstd = np.asarray(rstd, np.float64)[:, None]
    g, xh = dy * w, s * rstd
    dx = rstd * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    if ds is not None:
        dx = dx + np.asarray(ds, np.float64)
    return dx, np.sum(dy * xh, axis=0)
