"""fp64 selective state space scan: forward, step and gradients.

TEST INFRASTRUCTURE ONLY (see ``oracle/seq.py``).  Token by token from the definition;
``backward`` is reverse mode over the tokens (pinned by finite differences); with ``ckpt``
the states inside each block of 32 tokens start from the given ones.
"""
from __future__ import annotations

import numpy as np

from oracle.conv import silu

BLOCK = 32


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def time_step(dt, dt_bias=None, softplus=True):
    """(d, its slope, the pre-activation)."""
    pre = _f64(dt) + (0.0 if dt_bias is None else _f64(dt_bias))
    if not softplus:
        return pre, np.ones_like(pre), pre
    with np.errstate(over="ignore"):
        return np.logaddexp(pre, 0.0), 1.0 / (1.0 + np.exp(-pre)), pre


def spread(v, C):
    """[..., G, N] -> [..., C, N]."""
    return np.repeat(_f64(v), C // v.shape[-2], axis=-2)


def _live(lens, B, T):
    if lens is None:
        return np.ones((B, T), bool)
    return np.arange(T)[None] < np.clip(np.asarray(lens), 0, T)[:, None]


def pieces(x, dt, A, Bv, Cv, dt_bias=None, softplus=True, lens=None):
    """d, slope, pre, x, a, v, C of every token; tokens behind a row's end without effect."""
    x = _f64(x)
    B, T, C = x.shape
    d, slope, pre = time_step(dt, dt_bias, softplus)
    live = _live(lens, B, T)
    x, d = np.where(live[:, :, None], x, 0.0), np.where(live[:, :, None], d, 0.0)
    Bs = np.where(live[:, :, None, None], spread(Bv, C), 0.0)
    Cs = np.where(live[:, :, None, None], spread(Cv, C), 0.0)
    a = np.exp(d[..., None] * _f64(A))
    return dict(x=x, d=d, slope=slope, pre=pre, a=a, B=Bs, C=Cs, v=(d * x)[..., None] * Bs, live=live)


def _run(q, h, ckpt=None):
    """The states before each token, and the last one."""
    prev = np.empty_like(q["a"])
    for t in range(prev.shape[1]):
        if ckpt is not None and t % BLOCK == 0:
            h = np.swapaxes(_f64(ckpt)[:, t // BLOCK], 1, 2)
        prev[:, t] = h
        h = q["a"][:, t] * h + q["v"][:, t]
    return prev, h


def forward(x, dt, A, Bv, Cv, D=None, z=None, h0=None, **kw):
    """(y [B,T,C], h_T [B,C,N], block-start states [B,ceil(T/32),N,C])."""
    q = pieces(x, dt, A, Bv, Cv, **kw)
    B, T, C, N = q["a"].shape
    prev, h = _run(q, np.zeros((B, C, N)) if h0 is None else _f64(h0))
    u = ((q["a"] * prev + q["v"]) * q["C"]).sum(-1)
    if D is not None:
        u = u + _f64(D) * q["x"]
    y = u if z is None else u * silu(_f64(z))[0]
    return np.where(q["live"][:, :, None], y, 0.0), h, np.swapaxes(prev[:, ::BLOCK], 2, 3)


def step(h, x, dt, A, Bv, Cv, D=None, z=None, dt_bias=None, softplus=True):
    """(y [R,C], h [R,C,N])."""
    one = [np.asarray(t)[:, None] for t in (x, dt)]
    y, h, _ = forward(*one, A, np.asarray(Bv)[:, None], np.asarray(Cv)[:, None], D=D,
                      z=None if z is None else np.asarray(z)[:, None], h0=h, dt_bias=dt_bias, softplus=softplus)
    return y[:, 0], h


def backward(dy, x, dt, A, Bv, Cv, D=None, z=None, h0=None, ckpt=None, dh=None, **kw):
    """dict dx, ddt, dA, dB, dC, dD, dz, dbias, dh0, and the pieces the tolerances need."""
    q = pieces(x, dt, A, Bv, Cv, **kw)
    B, T, C, N = q["a"].shape
    G = np.asarray(Bv).shape[-2]
    prev, _ = _run(q, np.zeros((B, C, N)) if h0 is None else _f64(h0), ckpt)
    h = q["a"] * prev + q["v"]
    g0 = np.where(q["live"][:, :, None], _f64(dy), 0.0)
    u = (h * q["C"]).sum(-1) + (0.0 if D is None else _f64(D) * q["x"])
    out = dict(q=q, prev=prev, h=h, u=u, g0=g0)
    g = g0
    if z is not None:
        val, slope = silu(np.where(q["live"][:, :, None], _f64(z), 0.0))
        out["dz"] = g0 * u * slope
        g = g0 * val
    H = np.empty_like(h)
    K = np.zeros((B, C, N)) if dh is None else _f64(dh)
    for t in reversed(range(T)):
        H[:, t] = K + q["C"][:, t] * g[:, t, :, None]
        K = q["a"][:, t] * H[:, t]
    live = q["live"][:, :, None]
    qq = H * q["a"] * prev
    p = (H * q["B"]).sum(-1)
    dd = np.where(live, ((qq * _f64(A)).sum(-1) + p * q["x"]) * q["slope"], 0.0)
    dx = p * q["d"] + (0.0 if D is None else _f64(D) * g)

    def over_channels(t):
        return t.reshape(B, T, G, C // G, N).sum(3)
    out.update(dx=np.where(live, dx, 0.0), ddt=dd, dbias=dd.sum((0, 1)), dA=(qq * q["d"][..., None]).sum((0, 1)),
               dD=(g * q["x"]).sum((0, 1)), dB=over_channels(H * (q["d"] * q["x"])[..., None]),
               dC=over_channels(g[..., None] * h), dh0=K, H=H, p=p, qq=qq, g=g)
    return out
