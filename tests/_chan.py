"""Inputs and derived tolerances of the channelwise operators' GPU tests.

Every bound counts roundings.  E = 2^-24 is half a step of fp32 relative to the
value; a hardware exp, log, rcp or sqrt is off by at most a whole step (2 E).  An
output rounded to bf16 is off by 2^-8 of itself on top.
"""
import numpy as np

from synth.gen import bf16_round

E = 2.0 ** -24


def half_step(io):
    return 2.0 ** -8 if io == "bf16" else E


def dev(x, io=None):
    import torch
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.bfloat16() if io == "bf16" else t


def host(t):
    return t.double().cpu().numpy()


def check(name, got, want, tol):
    """|got - want| <= tol everywhere, both finite; reports the worst share of the bound."""
    got = host(got) if hasattr(got, "cpu") else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.all(np.isfinite(got)), name
    tol = np.broadcast_to(tol, want.shape) + 1e-37
    share = np.abs(got - want) / tol
    i = np.unravel_index(np.argmax(share), share.shape) if share.size else ()
    print(f"{name}: {share.max() if share.size else 0:.3f} of the bound", flush=True)
    assert share.size == 0 or share.max() <= 1.0, (name, i, got[i], want[i], tol[i])


# ---------------------------------------------------------------- the recurrence
def scan_inputs(lead, C, io, kind, seed, reset=False):
    """fp32 host arrays (values of ``io`` where the tensor has that type)."""
    rng = np.random.default_rng(seed)
    cast = bf16_round if io == "bf16" else (lambda z: z.astype(np.float32))

    def normal(*s):
        return rng.standard_normal(s).astype(np.float32)
    d = dict(x=cast(normal(*lead, C)), h=normal(lead[0], C), dy=cast(normal(*lead, C)), dh=normal(lead[0], C))
    if kind == "alpha":
        al = np.exp(-rng.uniform(0.01, 1, C) * np.log1p(np.exp(normal(*lead, C)))).astype(np.float32)
        if reset:
            al[rng.uniform(size=lead) < 0.05] = 0.0
            al[rng.uniform(size=lead) < 0.05] = 1.0
        d["kw"] = dict(alpha=al)
    else:
        dx = normal(*lead, C)
        if reset:                       # decays from 1 - 1e-8 to exp(-30)
            dx = dx * 8
        d["kw"] = dict(d=cast(dx), A=np.exp(rng.uniform(np.log(0.01), 0, C)).astype(np.float32),
                       normalise="norm" in kind)
        if "gate" in kind:
            d["kw"]["g"] = cast(normal(*lead, C) * (4 if reset else 1))
    return d


def gate_bounds(q, g):
    """Relative errors (in E) of a and of b from their evaluation in fp32.

    softplus: for d >= 0 it is at least ln 2, and w = e^-|d| enters it by less than its
    own size: exp, log and two additions, 8 E.  For d < 0 it is about w, whose exponent
    |d| log2 e is rounded once (E) from a constant that is off by 0.22 E: ln 2 |d| log2 e
    1.22 E = 1.22 |d| E on top, N = 1.3 |d| below.  u = A sp: 9 + N.  a = exp2(-u log2 e):
    the argument's relative error 11 + N moves a by (11 + N) u, the exp 2 E.  m = 1 - a^2:
    below z = 2u = 1/2 as z times a fit, whose error is z's, 9 + N, and at most 9 of its
    own (the fit 1.4, its evaluation); above, a^2's relative error 2 ((11 + N) u + 2) + 1
    divided by m >= 0.39 with a^2 <= 0.61.  (The bound changes over between z = 0.2 and
    0.3, where the second is the larger.)  b takes half of m's, 2 for the sqrt, 2 for
    products; the sigmoid 2 (|g| + 1) for its argument and exp, 1 for 1 + e, 2 for the
    rcp."""
    if q["u"] is None:
        return 0.0, 0.0
    u = q["u"]
    with np.errstate(divide="ignore"):
        d = np.log(q["sig"]) - np.log1p(-q["sig"])
    q["neg"] = 1.3 * np.where(d < 0, np.minimum(-d, 200.0), 0.0)
    ra = (11 + q["neg"]) * u + 2
    rb = np.zeros_like(u)
    if q["m"] is not None:
        series = 2 * u < 0.3
        with np.errstate(divide="ignore", invalid="ignore"):
            direct = (2 * ra + 1) * q["a"] ** 2 / q["m"] + 1
        q["rm"] = np.where(series, 18.0 + q["neg"], np.minimum(direct, 1e6))
        q["rm"] = np.where((2 * u > 0.2) & series, np.maximum(q["rm"], direct), q["rm"])
        rb = rb + q["rm"] / 2 + 4
    if q["s"] is not None:
        rb = rb + 2 * (np.abs(g) + 1) + 4
    return ra, rb


def scan_error(a, v, ra, rv, h0):
    """Bound of |error(h_t)| over the tokens, and of the state before each: every
    token rounds h once (E |h|) and, where a run of tokens is applied to a carried
    state at once, the run's product rounds once a token (2 E |a h|); the relative
    errors ra of a and rv of v enter where the values do."""
    B, T, C = v.shape
    M, N = np.abs(h0), np.zeros_like(h0)
    after, before = np.empty_like(v), np.empty_like(v)
    ra, rv = np.broadcast_to(ra, v.shape), np.broadcast_to(rv, v.shape)
    for t in range(T):
        before[:, t] = N
        N = a[:, t] * (N + (ra[:, t] + 2) * E * M) + rv[:, t] * E * np.abs(v[:, t])
        M = a[:, t] * M + np.abs(v[:, t])
        N = N + 2 * E * M
        after[:, t] = N
    return after, N, before


# ---------------------------------------------------------------- the norm
# Longest run of additions behind one row's sum: 65536 values over 256 threads,
# then the joins.
ROW_DEPTH = 256 + 16


def norm_bounds(x, w, mean, rstd, eps, y, io):
    """|errors| of y, mean and rstd."""
    D = x.shape[-1]
    dm = (min(D, ROW_DEPTH) + 2) * E * np.abs(x).sum(-1) / D
    # sum((x - m')^2) = sum((x - m)^2) + D dm^2; each square 4 E; eps, division, sqrt and rcp 8 E
    var = 1 / rstd ** 2
    c = x - mean[..., None]
    rr = ((min(D, ROW_DEPTH) + 5) * E + dm ** 2 / var + 2 * E * (np.abs(c).mean(-1) * np.abs(mean)) / var) / 2 + 8 * E
    wn = 1.0 if w is None else np.abs(w)
    dc = dm[..., None] + E * np.abs(c)
    dy = wn * (dc * rstd[..., None] + np.abs(c) * rstd[..., None] * (rr[..., None] + 4 * E)) + 2 * E * np.abs(y)
    xh = np.abs(c) * rstd[..., None] * wn
    return dy + 2 * E * xh + half_step(io) * np.abs(y), dm, rr * rstd


def norm_bwd_bounds(dy, x, mean, rstd, w, dx, xh, io):
    """|errors| of dx, dweight and dbias."""
    R, D = x.shape
    r = rstd[:, None]
    exh = E * (np.abs(x) + np.abs(mean[:, None])) * r + 3 * E * np.abs(xh)
    g = dy if w is None else dy * w
    ga = np.abs(g)
    n = min(D, ROW_DEPTH) + 4
    s1 = np.abs((g * xh).mean(-1, keepdims=True))
    e0 = n * E * ga.mean(-1, keepdims=True)
    e1 = n * E * (ga * np.abs(xh)).mean(-1, keepdims=True) + (ga * exh).mean(-1, keepdims=True)
    s0 = np.abs(g.mean(-1, keepdims=True))
    edx = r * (e0 + np.abs(xh) * e1 + s1 * exh + 6 * E * (ga + s0 + np.abs(xh) * s1))
    # the columns: at least 64 partial sums, at most 128 + R / 64 additions behind any value
    k = min(R, 128 + R // 64) + 4
    edw = (k * E * np.abs(dy * xh) + np.abs(dy) * exh).sum(0)
    edb = k * E * np.abs(dy).sum(0)
    return edx + half_step(io) * np.abs(dx), edw, edb
