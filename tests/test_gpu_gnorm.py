"""GPU parity of the gated group norm against the fp64 oracle, element by element."""
import itertools

import numpy as np
import pytest

from oracle import gnorm
from tests import _mixer as m

pytestmark = pytest.mark.gpu

# R, G, D: groups of less than a run, of every width a kernel has, of odd sizes
SHAPES = [(1, 1, 1), (3, 5, 2), (1, 16, 128), (700, 2, 3), (9, 7, 33), (513, 1, 64), (5, 3, 100), (2, 40, 17), (33, 2, 250),
          (4, 1, 511), (6, 2, 1000), (3, 1, 2049), (2, 1, 4097), (3, 2, 5000), (2, 1, 16384), (1, 1, 12289), (2000, 16, 8)]


def _inputs(R, G, D, io, seed):
    rng = np.random.default_rng(seed)
    f = m.cast(io)
    C = G * D

    def normal(*s):
        return rng.standard_normal(s).astype(np.float32)
    return dict(x=f(normal(R, C) + rng.standard_normal(1).astype(np.float32)), z=f(2 * normal(R, C)), w=normal(C), b=normal(C),
                dy=f(normal(R, C)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_forward_and_backward(i, shape, io):
    import recurrent_state_memory_amd as gdr
    R, G, D = shape
    d = _inputs(R, G, D, io, i)
    for k, (gate, act, center) in enumerate(itertools.product((False, True), repeat=3)):
        if i >= 6 and k % 4 != i % 4:          # all forms on the first shapes, two on each of the others
            continue
        z = d["z"] if gate else None
        kw = dict(z=m.dev(z, io), silu=act)
        # with eps of the size of the values, groups of one value have a mean square of their own
        eps = 1e-5 if D > 2 else 0.5
        y, mean, rstd = gdr.gdr_gnorm_fwd(m.dev(d["x"], io), G, m.dev(d["w"]), m.dev(d["b"]), center=center, eps=eps, **kw)
        y_r, m_r, r_r, u = gnorm.forward(d["x"], G, d["w"], d["b"], z, act, center, eps)
        ey, em, er = m.gnorm_fwd_bounds(d["x"], G, d["w"], d["b"], z, act, center, y_r, m_r, r_r, u, io)
        m.check("y", y, y_r, ey)
        m.check("rstd", rstd, r_r, er)
        assert (mean is None) == (not center)
        if center:
            m.check("mean", mean, m_r, em)
        g = gdr.gdr_gnorm_bwd(m.dev(d["dy"], io), m.dev(d["x"], io), mean, rstd, G, m.dev(d["w"]), m.dev(d["b"]), **kw)
        mh, rh = m.host(mean) if center else np.zeros_like(r_r), m.host(rstd)
        r = gnorm.backward(d["dy"], d["x"], mh, rh, G, d["w"], d["b"], z, act, center)
        ex, ez, ew, eb = m.gnorm_bwd_bounds(d["dy"], d["x"], mh, rh, G, d["w"], d["b"], z, act, center, r, io)
        m.check("dx", g["x"], r["dx"], ex)
        m.check("dw", g["weight"], r["dw"], ew)
        m.check("db", g["bias"], r["db"], eb)
        if gate:
            m.check("dz", g["z"], r["dz"], ez)


def test_optional_arguments():
    import torch
    import recurrent_state_memory_amd as gdr
    d = _inputs(6, 4, 24, "bf16", 3)
    x, dy = m.dev(d["x"], "bf16").view(2, 3, 96), m.dev(d["dy"], "bf16").view(2, 3, 96)
    one, zero = torch.ones(96, device="cuda"), torch.zeros(96, device="cuda")
    y, mean, rstd = gdr.gdr_gnorm_fwd(x, 4)
    assert mean.shape == rstd.shape == (2, 3, 4)
    y1, _, _ = gdr.gdr_gnorm_fwd(x, 4, one, zero)
    assert torch.equal(y, y1)
    y2, m2, r2 = gdr.gdr_gnorm_fwd(x, 4, return_stats=False, y=torch.empty_like(x))
    assert torch.equal(y, y2) and m2 is None and r2 is None
    g = gdr.gdr_gnorm_bwd(dy, x, mean, rstd, 4, one, zero)
    g1 = gdr.gdr_gnorm_bwd(dy, x, mean, rstd, 4, need_grad_weight=False)
    g2 = gdr.gdr_gnorm_bwd(dy, x, mean, rstd, 4, need_grad_weight=False, need_grad_bias=False)
    assert set(g1) == {"x", "bias"} and set(g2) == {"x"}
    assert torch.equal(g["x"], g1["x"]) and torch.equal(g["x"], g2["x"]) and torch.equal(g["bias"], g1["bias"])


def test_one_group_is_the_layer_norm():
    """With one group and neither gate nor activation the formulas are gdr_norm_fwd's."""
    import recurrent_state_memory_amd as gdr
    d = _inputs(50, 1, 300, "f32", 4)
    y, mean, rstd = gdr.gdr_gnorm_fwd(m.dev(d["x"]), 1, m.dev(d["w"]), m.dev(d["b"]))
    yn, mn, rn, _ = gdr.gdr_norm_fwd(m.dev(d["x"]), m.dev(d["w"]), m.dev(d["b"]))
    y_r, m_r, r_r, u = gnorm.forward(d["x"], 1, d["w"], d["b"])
    ey, em, er = m.gnorm_fwd_bounds(d["x"], 1, d["w"], d["b"], None, False, True, y_r, m_r, r_r, u, "f32")
    m.check("y", y, m.host(yn), 2 * ey)
    m.check("rstd", rstd[:, 0], m.host(rn), 2 * er[:, 0])


def test_rows_keep_to_themselves():
    """NaN and Inf stay within their group of their row; unaligned buffers keep their bounds."""
    import torch
    import recurrent_state_memory_amd as gdr
    R, G, D = 5, 3, 21
    d = _inputs(R, G, D, "bf16", 8)
    x, dy, w, b, z = (m.dev(d[k], io) for k, io in (("x", "bf16"), ("dy", "bf16"), ("w", None), ("b", None), ("z", "bf16")))
    y, mean, rstd = gdr.gdr_gnorm_fwd(x, G, w, b, z=z, silu=True)
    g = gdr.gdr_gnorm_bwd(dy, x, mean, rstd, G, w, b, z=z, silu=True)
    bad = x.clone()
    bad[2, 30], bad[4, 0] = float("nan"), float("inf")
    y1, mean1, rstd1 = gdr.gdr_gnorm_fwd(bad, G, w, b, z=z, silu=True)
    g1 = gdr.gdr_gnorm_bwd(dy, bad, mean1, rstd1, G, w, b, z=z, silu=True)
    hit = torch.zeros(R, G, D, dtype=torch.bool, device="cuda")
    hit[2, 1] = hit[4, 0] = True
    hit = hit.view(R, G * D)
    assert torch.equal(y1[~hit], y[~hit]) and torch.equal(g1["x"][~hit], g["x"][~hit])
    assert not bool(torch.isfinite(y1[hit]).any())
    n = x.numel()
    for off in (1, 5):
        buf = torch.full((n + 32,), 3.0, dtype=torch.bfloat16, device="cuda")
        src = torch.zeros(n + 32, dtype=torch.bfloat16, device="cuda")
        src[off:off + n] = x.flatten()
        o = buf[off:off + n].view(R, G * D)
        gdr.gdr_gnorm_fwd(src[off:off + n].view(R, G * D), G, w, b, z=z, silu=True, y=o)
        assert torch.equal(o, y) and bool((buf[:off] == 3).all()) and bool((buf[off + n:] == 3).all())
