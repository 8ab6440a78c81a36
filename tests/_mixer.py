"""Inputs and derived tolerances of the convolution's, the selective scan's and the gated
group norm's GPU tests.

Every bound counts roundings.  E = 2^-24 is half a step of fp32 relative to the value; a
hardware exp, rcp or log is off by at most a whole step (2 E).  An output rounded to bf16
is off by 2^-8 of itself on top.  A sum of n terms in any order is off by at most n E of
the sum of their magnitudes.
"""
import numpy as np

from oracle import conv, gnorm, ssm
from synth.gen import bf16_round
from tests._chan import E, ROW_DEPTH, check, dev, half_step, host  # noqa: F401


def cast(io):
    return bf16_round if io == "bf16" else (lambda z: np.asarray(z, np.float32))


def silu_err(v):
    """Relative error (in E) of silu(v) and of its slope's factors: the exponent's argument
    (2 |v|), exp, the addition and rcp 5, products 3."""
    return 2 * np.abs(v) + 8


# |slope of silu| <= 1.1; its evaluation s (1 + v (1 - s)): s relative 2 |v| + 5; 1 - s
# absolute (2 |v| + 6) E s; the rest 4 roundings of terms of at most 1 + |v|
def slope_err(v):
    return (2 * np.abs(v) + 6) * (1 + np.abs(v)) * 2 + 4 * (1 + np.abs(v))


def as_int32(lens):
    import torch
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- convolution
def conv_inputs(B, T, C, K, io, seed):
    rng = np.random.default_rng(seed)
    f = cast(io)

    def normal(*s):
        return rng.standard_normal(s).astype(np.float32)
    return dict(x=f(normal(B, T, C)), w=normal(C, K) * np.float32(0.5), b=normal(C), st=f(normal(B, K - 1, C)),
                dy=f(normal(B, T, C)), dst=f(normal(B, K - 1, C)))


def conv_bounds(d, K, act, y, u, io):
    """|error| of y: K fma on the bias, then the activation."""
    rows = np.concatenate([d["st"], d["x"]], 1).astype(np.float64)
    T = d["x"].shape[1]
    mag = sum(np.abs(d["w"][:, j] * rows[:, j:j + T]) for j in range(K)) + np.abs(d["b"])
    eu = (K + 1) * E * mag
    return eu, (1.1 * eu + silu_err(u) * E * np.abs(y) if act else eu) + half_step(io) * np.abs(y)


def conv_bwd_bounds(d, g, K, act, eu, io, parts):
    """|errors| of dx, dstate, dw, db; ``parts`` bounds the additions behind a weight's sum."""
    w, rows = np.abs(d["w"].astype(np.float64)), np.abs(g["rows"])
    T = d["x"].shape[1]
    dy = np.abs(d["dy"].astype(np.float64))
    # the slope's own slope is at most 0.5 + |u| / 4 < 1 + |u|
    ed = dy * ((1 + np.abs(g["u"])) * eu + slope_err(g["u"]) * E) + 2 * E * np.abs(g["d"]) if act else np.zeros_like(dy)
    ed = np.where(g["d"] == 0, 0, ed)
    grow = np.zeros_like(rows)
    for j in range(K):
        grow[:, j:j + T] += w[:, j] * (ed + (K + 1) * E * np.abs(g["d"]))
    grow = grow + 2 * E * 8 * np.abs(d["dst"]).max()
    full = np.concatenate([g["dstate"], g["dx"]], 1)
    out = grow + half_step(io) * np.abs(full)
    ew = np.stack([((ed + parts * E * np.abs(g["d"])) * rows[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
    eb = (ed + parts * E * np.abs(g["d"])).sum((0, 1))
    return out[:, K - 1:], out[:, :K - 1], ew, eb


# ---------------------------------------------------------------- selective scan
def ssm_inputs(B, T, C, N, G, io, seed, softplus=True, wild=False):
    rng = np.random.default_rng(seed)
    f = cast(io)

    def normal(*s):
        return rng.standard_normal(s).astype(np.float32)
    step = np.exp(rng.uniform(np.log(1e-3), np.log(0.1), C))
    if wild:     # time steps from 1e-4 to 40: from next to no decay to none of the state left
        step = np.exp(rng.uniform(np.log(1e-4), np.log(40.0), C))
    inv = (step + np.log(-np.expm1(-step))).astype(np.float32)
    d = dict(x=f(normal(B, T, C)), A=(-np.arange(1, N + 1) * np.exp(0.1 * normal(C, N))).astype(np.float32),
             Bv=f(normal(B, T, G, N)), Cv=f(normal(B, T, G, N)), D=normal(C), z=f(2 * normal(B, T, C)),
             h0=normal(B, C, N), dy=f(normal(B, T, C)), dh=normal(B, C, N), dt_bias=inv)
    d["dt"] = f(0.5 * normal(B, T, C))
    if not softplus:
        d["dt"] = f(step * np.exp(0.5 * normal(B, T, C)))
        d["dt_bias"] = np.zeros(C, np.float32)
    return d


def _step_err(q, softplus):
    """Relative error (in E) of d.  The sum dt + bias rounds once (|pre| slope absolute).
    softplus: 8 for its evaluation; below 0 the exponent's argument 1.3 |pre| on top."""
    if not softplus:
        return np.ones_like(q["d"])
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 8 + 1.3 * np.maximum(-q["pre"], 0) + np.abs(q["pre"]) * q["slope"] / q["d"]
    return np.where(q["live"][:, :, None], r, 0)


# An exponential below fp32's least normal number counts as 0: off by at most TINY, on top of
# its relative error, so whatever it multiplies (M, |H h|) adds TINY of itself.
TINY = 2.0 ** -126


def ssm_state_errors(q, h, prev, h0, ckpt, softplus):
    """Bounds of |error| of h_t and of the state before it, over the tokens.  a = exp2(d A2):
    the argument's relative error that of d and 3 more (A log2 e, its constant, the
    product) moves a by that many |d A|, exp2 2 E.  A run of tokens whose decay is taken at once
    (segments) uses the sum of their d, off by at most T/16 + 24 E of itself, which counts
    like an error of each d.  v = (d x) B: d's and 2; the fma 1."""
    B, T, C, N = q["a"].shape
    rd = _step_err(q, softplus)[..., None]
    with np.errstate(divide="ignore"):
        u = np.abs(np.log(np.maximum(q["a"], 1e-300)))
    ra = (rd + 3 + T / 16 + 24) * u + 3
    rv = rd + 3
    M = np.zeros((B, C, N)) if h0 is None else np.abs(np.asarray(h0, np.float64))
    Z = np.zeros((B, C, N))
    after, before, mag = np.empty_like(h), np.empty_like(h), np.empty_like(h)
    for t in range(T):
        if ckpt is not None and t % ssm.BLOCK == 0:
            M, Z = np.abs(prev[:, t]), np.zeros((B, C, N))
        before[:, t] = Z
        Z = q["a"][:, t] * (Z + ra[:, t] * E * M) + TINY * M + rv[:, t] * E * np.abs(q["v"][:, t])
        M = q["a"][:, t] * M + np.abs(q["v"][:, t])
        Z = Z + 2 * E * M
        after[:, t], mag[:, t] = Z, M
    return after, before, mag, ra, rd


def ssm_fwd_bounds(d, q, h, prev, y, io, softplus, gate, h0):
    after, before, mag, _, _ = ssm_state_errors(q, h, prev, h0, None, softplus)
    N = h.shape[-1]
    C = np.abs(q["C"])
    D = np.abs(d["D"]) * np.abs(q["x"])
    eu = (C * after).sum(-1) + (N + 10) * E * ((C * np.abs(h)).sum(-1) + D)
    if gate:
        z = d["z"].astype(np.float64)
        eu = eu * np.abs(conv.silu(z)[0]) + (silu_err(z) + 2) * E * np.abs(y)
    return eu + half_step(io) * np.abs(y), after[:, -1], before


def ssm_bwd_bounds(d, r, io, softplus, gate, h0, ckpt):
    """|errors| of every gradient, by name."""
    q, h, prev, H, g = r["q"], r["h"], r["prev"], r["H"], r["g"]
    B, T, C, N = h.shape
    after, before, _, ra, rd = ssm_state_errors(q, h, prev, h0, ckpt, softplus)
    z = np.where(q["live"][:, :, None], d["z"], 0.0)
    rg = silu_err(z) + 2 if gate else np.zeros_like(z)
    eg = rg * E * np.abs(g)
    Ca, Ba, a = np.abs(q["C"]), np.abs(q["B"]), q["a"]
    K, M = np.zeros((B, C, N)), np.abs(d["dh"].astype(np.float64))
    eH, mH = np.empty_like(h), np.empty_like(h)
    for t in reversed(range(T)):
        K = K + Ca[:, t] * eg[:, t, :, None]
        M = M + np.abs(q["C"][:, t] * g[:, t, :, None])
        K = K + 2 * E * M
        eH[:, t], mH[:, t] = K, M
        K = a[:, t] * (K + (ra[:, t] + 2) * E * M) + TINY * M
        M = a[:, t] * M
    dx = (q["d"] * q["x"])[..., None]
    xa, da = np.abs(q["x"]), np.abs(q["d"])
    qa = mH * a * np.abs(prev)
    eq = a * np.abs(prev) * (eH + (ra + 3) * E * mH) + mH * a * before + 3 * E * qa + TINY * mH * np.abs(prev)
    mp = (mH * Ba).sum(-1)
    ep = (eH * Ba).sum(-1) + (N + 10) * E * mp
    edx = ep * da + mp * da * (rd[..., 0] + 3) * E + np.abs(d["D"]) * (eg + 3 * E * np.abs(g))
    Aa = np.abs(d["A"].astype(np.float64))
    mdd = (Aa * qa).sum(-1) + mp * xa
    edd = (Aa * eq).sum(-1) + (N + 10) * E * (Aa * qa).sum(-1) + ep * xa + 3 * E * mdd
    # the slope of softplus: exp with its argument, two roundings, rcp; pre itself rounds
    rs = 2 * np.abs(q["pre"]) + 8 if softplus else 0.0
    edd = (edd + (rs + 1) * E * mdd) * q["slope"]
    out = dict(x=edx + half_step(io) * np.abs(r["dx"]), dt=edd + half_step(io) * np.abs(r["ddt"]))
    k = T + B + 64                                    # additions behind a parameter's sum
    out["A"] = (eq * da[..., None] + qa * da[..., None] * ((rd + 3) + k) * E).sum((0, 1))
    out["dt_bias"] = (edd + k * E * mdd * q["slope"]).sum((0, 1))
    out["D"] = ((eg + (k + 2) * E * np.abs(g)) * xa).sum((0, 1))
    out["h0"] = K + 2 * E * M
    G = d["Bv"].shape[2]
    n = C // G + 4

    def chans(t):
        return t.reshape(B, T, G, C // G, N).sum(3)
    out["B"] = chans((eH + (rd + 5 + n) * E * mH) * np.abs(dx)) + half_step(io) * np.abs(r["dB"])
    out["C"] = chans(eg[..., None] * np.abs(h) + np.abs(g)[..., None] * (after + (n + 2) * E * np.abs(h))) + \
        half_step(io) * np.abs(r["dC"])
    if gate:
        sl = conv.silu(z)[1]
        D = np.abs(d["D"]) * xa
        eu = (Ca * after).sum(-1) + (N + 10) * E * ((Ca * np.abs(h)).sum(-1) + D)
        g0 = np.abs(r["g0"])
        out["z"] = g0 * (eu * np.abs(sl) + np.abs(r["u"]) * (slope_err(z) + 4) * E) + half_step(io) * np.abs(r["dz"])
    return out


# ---------------------------------------------------------------- gated group norm
def _row_errors(x, mean, rstd, center):
    """|errors| of mean, of rstd (relative) and of xh, rows [R,G,D]."""
    D = x.shape[-1]
    depth = (min(D, ROW_DEPTH) + 5) * E
    dm = (min(D, ROW_DEPTH) + 2) * E * np.abs(x).sum(-1) / D if center else np.zeros(x.shape[:2])
    var = 1 / rstd ** 2
    c = x - mean[..., None]
    rr = (depth + dm ** 2 / var + 2 * E * (np.abs(c).mean(-1) * np.abs(mean)) / var) / 2 + 8 * E
    dc = dm[..., None] + E * np.abs(c)
    return dm, rr, dc * rstd[..., None] + np.abs(c) * rstd[..., None] * (rr[..., None] + 4 * E)


def gnorm_fwd_bounds(x, G, w, b, z, act, center, y, mean, rstd, u, io):
    R, C = x.shape
    xg = x.reshape(R, G, -1).astype(np.float64)
    dm, rr, eh = _row_errors(xg, mean, rstd, center)
    hat = np.abs((xg - mean[..., None]) * rstd[..., None]).reshape(R, C)
    eu = np.abs(w) * (eh.reshape(R, C) + 2 * E * hat) + E * (np.abs(w) * hat + np.abs(b))
    if z is not None:
        v = z.astype(np.float64)
        a = conv.silu(v)[0] if act else v
        ey = eu * np.abs(a) + (silu_err(v) if act else 1) * E * np.abs(y)
    else:
        ey = 1.1 * eu + silu_err(u) * E * np.abs(y) if act else eu
    return ey + half_step(io) * np.abs(y), dm, rr * rstd


def gnorm_bwd_bounds(dy, x, mean, rstd, G, w, b, z, act, center, r, io):
    """|errors| of dx, dz, dw, db; the statistics are the inputs' own."""
    R, C = x.shape
    D = C // G
    dy = np.abs(dy.astype(np.float64))
    hat, u = np.abs(r["xh"]), r["u"]
    spread = np.repeat(rstd, D, axis=1), np.repeat(np.abs(mean), D, axis=1)
    eh = E * (np.abs(x) + spread[1]) * spread[0] + 3 * E * hat
    wa = np.abs(w)
    eu = wa * eh + 2 * E * (wa * hat + np.abs(b))
    if z is not None:
        v = z.astype(np.float64)
        val, sl = conv.silu(v) if act else (v, np.ones_like(v))
        edu = (silu_err(v) if act else 1) * E * np.abs(r["du"]) + 2 * E * np.abs(r["du"])
        ez = dy * (eu * np.abs(sl) + np.abs(u) * ((slope_err(v) if act else 0) + 4) * E) + half_step(io) * np.abs(r["dz"])
    else:
        edu = dy * ((1 + np.abs(u)) * eu + slope_err(u) * E) + 2 * E * np.abs(r["du"]) if act else np.zeros_like(dy)
        ez = None
    g = (np.abs(r["du"]) * wa).reshape(R, G, D)
    eg = (edu * wa).reshape(R, G, D) + E * g
    h3, eh3 = hat.reshape(R, G, D), eh.reshape(R, G, D)
    n = min(D, ROW_DEPTH) + 6
    s0, s1 = g.mean(-1, keepdims=True), (g * h3).mean(-1, keepdims=True)
    e0 = eg.mean(-1, keepdims=True) + n * E * s0
    e1 = (eg * h3 + g * eh3).mean(-1, keepdims=True) + n * E * s1
    edx = eg + (e0 if center else 0) + h3 * e1 + eh3 * s1 + 6 * E * (g + s0 + h3 * s1)
    edx = (edx * rstd[..., None]).reshape(R, C) + half_step(io) * np.abs(r["dx"])
    k = min(R, 2048) + 80                             # rows behind a column's sum, and the joins
    ew = ((edu + k * E * np.abs(r["du"])) * hat + np.abs(r["du"]) * eh).sum(0)
    eb = (edu + k * E * np.abs(r["du"])).sum(0)
    return edx, ez, ew, eb
