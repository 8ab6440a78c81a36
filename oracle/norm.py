"""fp64 layer norm and its gradients.

TEST INFRASTRUCTURE ONLY (see ``oracle/seq.py``).  Pinned by finite differences.
"""
from __future__ import annotations

import numpy as np


def forward(x, weight=None, bias=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    c = x - mean[..., None]
    rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
    y = c * rstd[..., None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def backward(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias, xh) of rows [R,D] with the given statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * r
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = r * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh
