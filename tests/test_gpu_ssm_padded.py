"""The selective scan on padded batches whose rows are cut into segments (a row may end in any
of them, on the border of two, or one token behind it), and on batches of many rows that are
not cut, over many tiles, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import ssm
from tests import _mixer as m

pytestmark = pytest.mark.gpu


def _compare(B, T, C, N, G, io, lens, seed, softplus=True, gate=True, kept=(False, True)):
    import recurrent_state_memory_amd as gdr
    d = m.ssm_inputs(B, T, C, N, G, io, seed, softplus)
    t = {k: m.dev(d[k], io) for k in ("x", "dt", "Bv", "Cv", "z", "dy")}
    for b, n in enumerate(lens or []):          # nothing behind a row's end is read
        for k in t:
            t[k][b, n:] = float("nan")
    args = (t["x"], t["dt"], m.dev(d["A"]), t["Bv"], t["Cv"])
    kw = dict(D=m.dev(d["D"]), z=t["z"] if gate else None, dt_bias=m.dev(d["dt_bias"]), softplus=softplus, lens=m.as_int32(lens))
    ref = dict(D=d["D"], z=d["z"] if gate else None, dt_bias=d["dt_bias"], softplus=softplus, lens=lens)
    ins = (d["x"], d["dt"], d["A"], d["Bv"], d["Cv"])
    y, h, ck = gdr.gdr_ssm_fwd(*args, h0=m.dev(d["h0"]), return_ckpt=True, **kw)
    r = ssm.backward(d["dy"], *ins, h0=d["h0"], dh=d["dh"], **ref)
    y_r, h_r, ck_r = ssm.forward(*ins, h0=d["h0"], **ref)
    ey, eh, before = m.ssm_fwd_bounds(d, r["q"], r["h"], r["prev"], y_r, io, softplus, gate, d["h0"])
    m.check("y", y, y_r, ey)
    m.check("h", h, h_r, eh)
    m.check("ckpt", ck, ck_r, np.swapaxes(before[:, ::32], 2, 3))
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", h0="dh0", D="dD", dt_bias="dbias")
    names.update({"z": "dz"} if gate else {})
    for k in kept:
        ckh = m.host(ck) if k else None
        g = gdr.gdr_ssm_bwd(t["dy"], *args, h0=None if k else m.dev(d["h0"]), ckpt=ck if k else None, grad_h=m.dev(d["dh"]), **kw)
        if k:
            r = ssm.backward(d["dy"], *ins, ckpt=ckh, dh=d["dh"], **ref)
        e = m.ssm_bwd_bounds(d, r, io, softplus, gate, d["h0"], ckh)
        assert set(g) == set(names)
        for name, rk in names.items():
            m.check("d" + name, g[name], r[rk], e[name])


# Forward: 12 chains of 700 tokens in 8 segments of 96, 14 of 600 in 7 of 96, 5 of 515 in 6 of 96.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,N,G,lens", [
    (6, 700, 66, 16, 1, [37, 96, 97, 350, 690, 700]), (7, 600, 40, 40, 2, [0, 1, 95, 192, 193, 577, 599]),
    (5, 515, 5, 3, 1, [300, 480, 481, 32, 515]), (1, 1500, 20, 33, 2, [800]), (1, 900, 64, 16, 1, [1]),
    (2, 400, 10, 8, 1, [0, 0])])
def test_rows_that_end_inside_a_segment(B, T, C, N, G, lens, io):
    _compare(B, T, C, N, G, io, lens, 100 + T, softplus=N != 3, gate=N != 16)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,N,padded", [(256, 330, 2, 16, False), (256, 290, 3, 5, True), (132, 420, 2, 20, True)])
def test_rows_of_many_tiles_that_are_not_cut(B, T, C, N, padded, io):
    """As in a layer's batch: enough chains of channels that each walks its row alone."""
    _compare(B, T, C, N, 1, io, [T - (b * 37) % (T + 1) for b in range(B)] if padded else None, 200 + T, kept=(N == 5,))
