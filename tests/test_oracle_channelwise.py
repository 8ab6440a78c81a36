"""Pins of the channelwise oracles: hand-computed values, finite differences of
every gradient, and the 8-bit codes against torch's own conversion."""
import numpy as np
import pytest

from oracle import ckpt8, norm, scan


def test_scan_by_hand():
    """a = 1/2 and 0, b = 1: h = 1, 2.5, 4 (reset), then the step."""
    x = np.array([1.0, 2.0, 4.0]).reshape(1, 3, 1)
    alpha = np.array([0.5, 0.5, 0.0]).reshape(1, 3, 1)
    y, h, ck = scan.forward(x, alpha=alpha)
    assert y.ravel().tolist() == [1.0, 2.5, 4.0] and h.ravel().tolist() == [4.0]
    assert ck.shape == (1, 1, 1) and ck[0, 0, 0] == 0.0
    assert scan.step(np.array([[2.0]]), np.array([[3.0]]), alpha=np.array([[0.25]]))[0, 0] == 3.5


def test_scan_gates_by_hand():
    """d = 0, A = 1: u = ln 2, a = 1/2, 1 - a^2 = 3/4; g = 0: sigmoid = 1/2."""
    q = scan.gates(d=np.zeros((1, 1)), A=np.ones(1), g=np.zeros((1, 1)), normalise=True)
    assert abs(q["a"][0, 0] - 0.5) < 1e-15 and abs(q["b"][0, 0] - 0.5 * np.sqrt(0.75)) < 1e-15


def _num(f, x, eps=1e-6):
    g = np.empty_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        hi = f()
        x[i] = old - eps
        lo = f()
        x[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("kind", ["alpha", "decay", "gate", "norm", "gate+norm"])
def test_scan_gradients_by_differences(kind):
    rng = np.random.default_rng(5)
    B, T, C = 2, 35, 2
    x, h0 = rng.standard_normal((B, T, C)), rng.standard_normal((B, C))
    dy, dh = rng.standard_normal((B, T, C)), rng.standard_normal((B, C))
    if kind == "alpha":
        kw = dict(alpha=rng.uniform(0, 1, (B, T, C)))
    else:
        kw = dict(d=rng.standard_normal((B, T, C)), A=rng.uniform(0.1, 1, C), normalise="norm" in kind)
        if "gate" in kind:
            kw["g"] = rng.standard_normal((B, T, C))

    def loss():
        y, h, _ = scan.forward(x, h0=h0, **kw)
        return (y * dy).sum() + (h * dh).sum()
    r = scan.backward(x, dy, dh, h0=h0, **kw)
    for name, arr in [("dx", x), ("dh0", h0), ("dalpha", kw.get("alpha")), ("dd", kw.get("d")), ("dA", kw.get("A")),
                      ("dg", kw.get("g"))]:
        if arr is not None:
            assert np.allclose(r[name], _num(loss, arr), rtol=1e-6, atol=1e-7), name
    # starting each block from the forward's own states changes nothing
    ck = scan.forward(x, h0=h0, **kw)[2]
    r2 = scan.backward(x, dy, dh, ckpt=ck, **kw)
    assert all(np.array_equal(r[k], r2[k]) for k in ("dx", "dh0"))


def test_norm_by_hand_and_differences():
    y, m, r = norm.forward(np.array([[1.0, 3.0]]), np.array([2.0, 2.0]), np.array([1.0, 0.0]), eps=0.0)
    assert y.tolist() == [[-1.0, 2.0]] and m.tolist() == [2.0] and r.tolist() == [1.0]
    rng = np.random.default_rng(6)
    x, w, b, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal(7), rng.standard_normal((3, 7))

    def loss():
        return (norm.forward(x, w, b)[0] * dy).sum()
    _, mean, rstd = norm.forward(x, w, b)
    dx, dw, db, _ = norm.backward(dy, x, mean, rstd, w)
    for got, arr in [(dx, x), (dw, w), (db, b)]:
        assert np.allclose(got, _num(loss, arr), rtol=1e-6, atol=1e-7)


def test_ckpt8_codes():
    import torch
    # every finite code is its own value under scale 1 (a 448 in each group)
    c = np.arange(256, dtype=np.uint8)
    c = c[(c & 127) != 127].reshape(2, 127)
    code, exp = ckpt8.pack(ckpt8.value(c, np.full((2, 1), 127)))
    assert np.array_equal(code, c) and np.all(exp == 127)
    # nearest, ties to even, against torch's conversion
    rng = np.random.default_rng(7)
    x = np.concatenate([rng.standard_normal((4, 200)) * 10.0 ** rng.uniform(-3, 3, (4, 1)),
                        np.full((4, 1), 0.0)], 1).astype(np.float32)
    code, exp = ckpt8.pack(x)
    E = np.repeat(exp.astype(np.float64), 128, 1)[:, :201]
    t = torch.from_numpy((x * 2.0 ** (127 - E)).astype(np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(t.view(torch.uint8).numpy(), code)
    for r in range(4):
        for j, g in enumerate((x[r, :128], x[r, 128:])):
            top = np.abs(g).max().astype(np.float64)
            assert top <= 448 * 2.0 ** (int(exp[r, j]) - 127) and (top > 448 * 2.0 ** (int(exp[r, j]) - 128))
    # no finite value, and a value too small for any code
    code, exp = ckpt8.pack(np.array([[np.inf, -np.inf, np.nan], [0.0, -0.0, 1e-42]]))
    assert code.tolist() == [[127, 255, 127], [0, 128, 0]] and exp.tolist() == [[1], [1]]
