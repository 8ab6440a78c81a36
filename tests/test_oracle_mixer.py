"""Pins of the convolution's, the selective scan's and the gated group norm's oracles."""
import numpy as np
import pytest

from oracle import conv, gnorm, ssm


def grad(f, x, eps=1e-6):
    x = np.array(x, np.float64)
    g = np.empty_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f(x)
        x[i] = keep - eps
        g[i] = (up - f(x)) / (2 * eps)
        x[i] = keep
    return g


def close(a, b, tol=2e-7):
    assert a.shape == b.shape
    assert np.max(np.abs(a - b), initial=0.0) <= tol * max(1.0, np.max(np.abs(b), initial=0.0)), np.max(np.abs(a - b))


def test_conv_by_hand():
    x = np.array([[[1.0], [2.0], [3.0]]])
    y, st, _ = conv.forward(x, np.array([[10.0, 1.0]]), np.array([0.5]), state=np.array([[[7.0]]]), act=False)
    assert y[0, :, 0].tolist() == [71.5, 12.5, 23.5] and st[0, 0, 0] == 3.0
    y, st, _ = conv.forward(x, np.array([[100.0, 10.0, 1.0]]), state=np.array([[[7.0], [8.0]]]), lens=[1], act=False)
    assert y[0, :, 0].tolist() == [781.0, 0.0, 0.0] and st[0, :, 0].tolist() == [8.0, 1.0]


def test_conv_is_numpys():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((1, 20, 3)), rng.standard_normal((3, 4))
    y, _, _ = conv.forward(x, w, act=False)
    for c in range(3):
        close(y[0, :, c], np.convolve(x[0, :, c], w[c, ::-1])[:20])


@pytest.mark.parametrize("act", [False, True])
def test_conv_gradients(act):
    rng = np.random.default_rng(1)
    B, T, C, K, lens = 3, 5, 2, 4, [5, 2, 0]
    x, w, b, st = (rng.standard_normal(s) for s in ((B, T, C), (C, K), (C,), (B, K - 1, C)))
    dy, ds = rng.standard_normal((B, T, C)), rng.standard_normal((B, K - 1, C))

    def loss(x=x, w=w, b=b, st=st):
        y, so, _ = conv.forward(x, w, b, st, lens, act)
        return (y * dy).sum() + (so * ds).sum()
    g = conv.backward(dy, x, w, b, st, lens, act, ds)
    close(g["dx"], grad(lambda v: loss(x=v), x))
    close(g["dw"], grad(lambda v: loss(w=v), w))
    close(g["db"], grad(lambda v: loss(b=v), b))
    close(g["dstate"], grad(lambda v: loss(st=v), st))


def test_ssm_by_hand():
    """One state and no time step: nothing is forgotten or written; with d = ln 2 and A = -1
    half of the state is left."""
    h0 = np.array([[[3.0]]])
    z = np.zeros((1, 1, 1))
    y, h, _ = ssm.forward(z + 5, z, [[-1.0]], z[..., None] + 2, z[..., None] + 4, h0=h0, softplus=False)
    assert y[0, 0, 0] == 12.0 and h[0, 0, 0] == 3.0
    y, h, _ = ssm.forward(z + 5, z + np.log(2), [[-1.0]], z[..., None] + 2, z[..., None] + 4, D=[1.0], h0=h0, softplus=False)
    close(h, np.array([[[1.5 + 10 * np.log(2)]]]))
    close(y, 4 * (1.5 + 10 * np.log(2)) + z + 5)
    assert ssm.time_step(np.zeros(1))[0][0] == np.log(2)


def test_ssm_groups_and_pieces():
    """Channels see their group's vectors; a call on each half gives the call on the whole."""
    rng = np.random.default_rng(2)
    B, T, C, N, G = 2, 70, 6, 3, 2
    x, dt = rng.standard_normal((B, T, C)), rng.standard_normal((B, T, C))
    A, Bv, Cv = -rng.uniform(0.1, 2, (C, N)), rng.standard_normal((B, T, G, N)), rng.standard_normal((B, T, G, N))
    y, h, ck = ssm.forward(x, dt, A, Bv, Cv)
    y1, h1, _ = ssm.forward(x[..., 3:], dt[..., 3:], A[3:], Bv[:, :, 1:], Cv[:, :, 1:])
    close(y[..., 3:], y1)
    ya, ha, _ = ssm.forward(x[:, :64], dt[:, :64], A, Bv[:, :64], Cv[:, :64])
    close(np.swapaxes(ha, 1, 2), ck[:, 2])
    yb, hb, _ = ssm.forward(x[:, 64:], dt[:, 64:], A, Bv[:, 64:], Cv[:, 64:], h0=ha)
    close(np.concatenate([ya, yb], 1), y)
    close(hb, h)
    ys, hs = ssm.step(ha, x[:, 64], dt[:, 64], A, Bv[:, 64], Cv[:, 64])
    close(ys, y[:, 64])


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_ssm_gradients(softplus, gate):
    rng = np.random.default_rng(3)
    B, T, C, N, G, lens = 3, 4, 4, 2, 2, [4, 2, 0]
    p = dict(x=rng.standard_normal((B, T, C)), dt=rng.uniform(0.1, 1, (B, T, C)), A=-rng.uniform(0.2, 2, (C, N)),
             Bv=rng.standard_normal((B, T, G, N)), Cv=rng.standard_normal((B, T, G, N)), D=rng.standard_normal(C),
             z=rng.standard_normal((B, T, C)) if gate else None, dt_bias=rng.standard_normal(C) * 0.1,
             h0=rng.standard_normal((B, C, N)))
    dy, dh = rng.standard_normal((B, T, C)), rng.standard_normal((B, C, N))

    def loss(**kw):
        y, h, _ = ssm.forward(**{**p, **kw}, softplus=softplus, lens=lens)
        return (y * dy).sum() + (h * dh).sum()
    g = ssm.backward(dy, dh=dh, softplus=softplus, lens=lens, **p)
    for name, key in [("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bv", "dB"), ("Cv", "dC"), ("D", "dD"), ("dt_bias", "dbias"),
                      ("h0", "dh0")] + [("z", "dz")] * gate:
        close(g[key], grad(lambda v: loss(**{name: v}), p[name]))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("center", [False, True])
def test_gnorm_gradients(gate, act, center):
    rng = np.random.default_rng(4)
    R, G, C = 3, 2, 10
    p = dict(x=rng.standard_normal((R, C)), weight=rng.standard_normal(C), bias=rng.standard_normal(C),
             z=rng.standard_normal((R, C)) if gate else None)
    dy = rng.standard_normal((R, C))

    def loss(**kw):
        q = {**p, **kw}
        return (gnorm.forward(q["x"], G, q["weight"], q["bias"], q["z"], act, center)[0] * dy).sum()
    _, mean, rstd, _ = gnorm.forward(p["x"], G, center=center)
    g = gnorm.backward(dy, p["x"], mean, rstd, G, p["weight"], p["bias"], p["z"], act, center)
    for name, key in [("x", "dx"), ("weight", "dw"), ("bias", "db")] + [("z", "dz")] * gate:
        close(g[key], grad(lambda v: loss(**{name: v}), p[name]), 1e-6)
    y, m, r, _ = gnorm.forward(np.array([[1.0, 3.0, 5.0, 9.0]]), 2, eps=0.0)
    assert m.tolist() == [[2.0, 7.0]] and r.tolist() == [[1.0, 0.5]] and y[0, :2].tolist() == [-1.0, 1.0]
