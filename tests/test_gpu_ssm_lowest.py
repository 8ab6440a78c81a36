"""The selective scan with decay rates that are held to -2^64, down to fp32's lowest value and
-Inf: such a state forgets all of its past at every token, and a time step of 0 still leaves
it alone."""
import numpy as np
import pytest

from oracle import ssm
from tests import _mixer as m

pytestmark = pytest.mark.gpu

LOW, HELD = np.float32(-3e38), np.float32(-2.0 ** 64)


def _inputs(B, T, C, N, io, seed):
    """Some states of every channel, and some whole channels, with the lowest rate."""
    d = m.ssm_inputs(B, T, C, N, 1, io, seed)
    d["A"][:, 1::3] = LOW
    d["A"][C // 2:] = LOW
    d["A"][C // 3] = -np.inf
    return d


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,N", [(2, 37, 66, 16), (3, 50, 40, 5), (1, 45, 70, 33), (2, 600, 20, 16), (2, 300, 64, 8)])
def test_forward_and_backward(B, T, C, N, io):
    """Rows that end inside a tile.  A time step is at least 1e-4 here, so those states' decays
    are 0 in the formula of the held rate and in fp32 alike, and the general bounds hold."""
    import recurrent_state_memory_amd as gdr
    d = _inputs(B, T, C, N, io, T + N)
    lens = [T, T // 2 + 3, 9][:B]
    t = {k: m.dev(d[k], io) for k in ("x", "dt", "Bv", "Cv", "z", "dy")}
    args = (t["x"], t["dt"], m.dev(d["A"]), t["Bv"], t["Cv"])
    kw = dict(D=m.dev(d["D"]), z=t["z"], dt_bias=m.dev(d["dt_bias"]), lens=m.as_int32(lens))
    ref = dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], lens=lens)
    d["A"] = np.maximum(d["A"], HELD)
    ins = (d["x"], d["dt"], d["A"], d["Bv"], d["Cv"])
    y, h, ck = gdr.gdr_ssm_fwd(*args, h0=m.dev(d["h0"]), return_ckpt=True, **kw)
    r = ssm.backward(d["dy"], *ins, h0=d["h0"], **ref)
    y_r, h_r, ck_r = ssm.forward(*ins, h0=d["h0"], **ref)
    ey, eh, before = m.ssm_fwd_bounds(d, r["q"], r["h"], r["prev"], y_r, io, True, True, d["h0"])
    m.check("y", y, y_r, ey)
    m.check("h", h, h_r, eh)
    m.check("ckpt", ck, ck_r, np.swapaxes(before[:, ::32], 2, 3))
    for kept in (False, True):
        ckh = m.host(ck) if kept else None
        g = gdr.gdr_ssm_bwd(t["dy"], *args, h0=None if kept else m.dev(d["h0"]), ckpt=ck if kept else None,
                            grad_h=m.dev(d["dh"]), **kw)
        r = ssm.backward(d["dy"], *ins, h0=d["h0"], ckpt=ckh, dh=d["dh"], **ref)
        e = m.ssm_bwd_bounds(d, r, io, True, True, d["h0"], ckh)
        for k, rk in dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", h0="dh0", D="dD", z="dz", dt_bias="dbias").items():
            m.check("d" + k, g[k], r[rk], e[k])


@pytest.mark.parametrize("N", [3, 16, 40])
def test_single_tokens(N):
    """A time step of exactly 0 leaves the state alone at any rate; others forget all of it."""
    import torch
    import recurrent_state_memory_amd as gdr
    R, C = 3, 70
    d = m.ssm_inputs(R, 1, C, N, 1, "f32", N, softplus=False)
    d["A"][:] = LOW
    d["A"][5], d["A"][6] = -np.inf, np.finfo(np.float32).min
    dt = d["dt"][:, 0].copy()
    dt[:, ::2] = 0
    h, x, Bv = m.dev(d["h0"]), m.dev(d["x"][:, 0]), m.dev(d["Bv"][:, 0])
    out = torch.empty_like(h)
    gdr.gdr_ssm_step(h, x, m.dev(dt), m.dev(d["A"]), Bv, m.dev(d["Cv"][:, 0]), softplus=False, h_out=out)
    assert torch.equal(out[:, ::2], h[:, ::2])
    assert torch.equal(out[:, 1::2], ((m.dev(dt) * x)[:, :, None] * Bv)[:, 1::2])
