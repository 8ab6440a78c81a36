"""fp64 short causal convolution: forward, step and gradients.

TEST INFRASTRUCTURE ONLY (see ``oracle/seq.py``).  Pinned by hand-computed values,
``numpy.convolve`` and finite differences.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def silu(v):
    """(v sigmoid(v), its slope)."""
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-v))
    return v * s, s * (1.0 + v * (1.0 - s))


def _rows(x, K, state):
    x = _f64(x)
    B, T, C = x.shape
    edge = np.zeros((B, K - 1, C)) if state is None else _f64(state)
    return np.concatenate([edge, x], 1)


def _ends(x, lens):
    B, T, _ = x.shape
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]


def forward(x, weight, bias=None, state=None, lens=None, act=True):
    """(y [B,T,C], state_out [B,K-1,C], u)."""
    w = _f64(weight)
    K = w.shape[1]
    rows = _rows(x, K, state)
    T = rows.shape[1] - K + 1
    u = sum(w[:, j] * rows[:, j:j + T] for j in range(K))
    if bias is not None:
        u = u + _f64(bias)
    y = silu(u)[0] if act else u.copy()
    ends = _ends(np.asarray(x), lens)
    for b, e in enumerate(ends):
        y[b, e:] = 0.0
    return y, np.stack([rows[b, e:e + K - 1] for b, e in enumerate(ends)]), u


def backward(dy, x, weight, bias=None, state=None, lens=None, act=True, dstate=None):
    """dict dx, dw, db, dstate, and d (the gradient of u)."""
    w = _f64(weight)
    C, K = w.shape
    rows = _rows(x, K, state)
    u = forward(x, weight, bias, state, None, False)[2]
    d = _f64(dy) * (silu(u)[1] if act else 1.0)
    T = d.shape[1]
    grow = np.zeros_like(rows)
    for b, e in enumerate(_ends(np.asarray(x), lens)):
        d[b, e:] = 0.0
        if dstate is not None:
            grow[b, e:e + K - 1] += _f64(dstate)[b]
    dw = np.empty((C, K))
    for j in range(K):
        grow[:, j:j + T] += w[:, j] * d
        dw[:, j] = (d * rows[:, j:j + T]).sum((0, 1))
    return dict(dx=grow[:, K - 1:], dstate=grow[:, :K - 1], dw=dw, db=d.sum((0, 1)), d=d, u=u, rows=rows)
