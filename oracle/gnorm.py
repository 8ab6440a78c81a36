"""fp64 group norm with its activation or gate, and its gradients.

TEST INFRASTRUCTURE ONLY (see ``oracle/seq.py``).  Pinned by finite differences.
"""
from __future__ import annotations

import numpy as np

from oracle.conv import silu


def _parts(x, G, mean, rstd, weight, bias):
    R, C = x.shape
    xh = ((x.reshape(R, G, -1) - mean[..., None]) * rstd[..., None]).reshape(R, C)
    u = xh * (1.0 if weight is None else np.asarray(weight, np.float64))
    return xh, u if bias is None else u + np.asarray(bias, np.float64)


def statistics(x, G, center=True, eps=1e-5):
    g = np.asarray(x, np.float64).reshape(x.shape[0], G, -1)
    mean = g.mean(-1) if center else np.zeros(g.shape[:2])
    c = g - mean[..., None]
    return mean, 1.0 / np.sqrt((c * c).mean(-1) + eps)


def forward(x, G, weight=None, bias=None, z=None, act=False, center=True, eps=1e-5):
    """(y [R,C], mean [R,G], rstd [R,G], u)."""
    x = np.asarray(x, np.float64)
    mean, rstd = statistics(x, G, center, eps)
    u = _parts(x, G, mean, rstd, weight, bias)[1]
    v = u if z is None else np.asarray(z, np.float64)
    a = silu(v)[0] if act else v
    return (a if z is None else u * a), mean, rstd, u


def backward(dy, x, mean, rstd, G, weight=None, bias=None, z=None, act=False, center=True):
    """dict dx, dz, dw, db and the pieces the tolerances need, with the given statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    R, C = x.shape
    mean, rstd = np.asarray(mean, np.float64), np.asarray(rstd, np.float64)
    xh, u = _parts(x, G, mean, rstd, weight, bias)
    v = u if z is None else np.asarray(z, np.float64)
    val, slope = silu(v) if act else (v, np.ones_like(v))
    du = dy * slope if z is None else dy * val
    out = dict(dw=(du * xh).sum(0), db=du.sum(0), xh=xh, u=u, du=du, dz=None if z is None else dy * u * slope)
    g = (du if weight is None else du * np.asarray(weight, np.float64)).reshape(R, G, -1)
    h = xh.reshape(R, G, -1)
    dx = g - h * (g * h).mean(-1, keepdims=True)
    if center:
        dx = dx - g.mean(-1, keepdims=True)
    out["dx"] = (dx * rstd[..., None]).reshape(R, C)
    return out
