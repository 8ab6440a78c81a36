"""fp64 channelwise gated linear recurrence: forward, step and gradients.

TEST INFRASTRUCTURE ONLY (see ``oracle/seq.py``).

Per batch row, channel and token: h_t = a_t h_{t-1} + b_t x_t, y_t = h_t, with
a = alpha, b = 1, or u = A softplus(d), a = exp(-u), b = [sigmoid(g)]
[sqrt(1 - a^2)].  ``backward`` is reverse mode over the tokens (pinned by finite
differences in the tests); with ``ckpt`` the states inside each block of 32
tokens start from the given ones, which is what a pass over an 8-bit copy of x
computes.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def gates(alpha=None, d=None, A=None, g=None, normalise=False):
    """dict of a, b and their makings (u, sp, s, m), broadcast over [...,C]."""
    if alpha is not None:
        a = _f64(alpha)
        return dict(a=a, b=np.ones_like(a), s=None, m=None, u=None, sp=None, sig=None)
    d = _f64(d)
    sp = np.logaddexp(d, 0.0)
    u = _f64(A) * sp
    a = np.exp(-u)
    s = None if g is None else 1.0 / (1.0 + np.exp(-_f64(g)))
    m = -np.expm1(-2.0 * u) if normalise else None
    b = np.ones_like(a)
    if s is not None:
        b = b * s
    if m is not None:
        b = b * np.sqrt(m)
    return dict(a=a, b=b, s=s, m=m, u=u, sp=sp, sig=1.0 / (1.0 + np.exp(-d)))


def forward(x, h0=None, **kw):
    """(y [B,T,C], h_T [B,C], block-start states [B,ceil(T/32),C])."""
    x = _f64(x)
    B, T, C = x.shape
    q = gates(**kw)
    h = np.zeros((B, C)) if h0 is None else _f64(h0).copy()
    y, ck = np.empty_like(x), np.empty((B, -(-T // BLOCK), C))
    for t in range(T):
        if t % BLOCK == 0:
            ck[:, t // BLOCK] = h
        h = q["a"][:, t] * h + q["b"][:, t] * x[:, t]
        y[:, t] = h
    return y, h, ck


def step(h, x, **kw):
    q = gates(**kw)
    return q["a"] * _f64(h) + q["b"] * _f64(x)


def backward(x, dy, dh=None, h0=None, ckpt=None, A=None, **kw):
    """dict dx, dalpha | (dd, dA, dg), dh0, and the pieces the tolerances need."""
    x, dy = _f64(x), _f64(dy)
    B, T, C = x.shape
    q = gates(A=A, **kw)
    a, b = q["a"], q["b"]
    h = np.zeros((B, C)) if h0 is None else _f64(h0).copy()
    prev = np.empty_like(x)
    for t in range(T):
        if ckpt is not None and t % BLOCK == 0:
            h = _f64(ckpt)[:, t // BLOCK]
        prev[:, t] = h
        h = a[:, t] * h + b[:, t] * x[:, t]
    G = np.empty_like(x)
    K = np.zeros((B, C)) if dh is None else _f64(dh).copy()
    for t in reversed(range(T)):
        G[:, t] = dy[:, t] + K
        K = a[:, t] * G[:, t]
    out = dict(dx=G * b, dh0=K, G=G, prev=prev, q=q)
    if q["u"] is None:
        out["dalpha"] = G * prev
        return out
    if q["s"] is not None:
        out["dg"] = G * b * x * (1.0 - q["s"])
    inner = -prev
    if q["m"] is not None:
        with np.errstate(divide="ignore", invalid="ignore"):
            inner = inner + np.where(q["m"] > 0, b * x * a / q["m"], 0.0)
    du = G * a * inner
    out["du"] = du
    out["dd"] = du * _f64(A) * q["sig"]
    out["dA"] = (du * q["sp"]).sum((0, 1))
    return out
