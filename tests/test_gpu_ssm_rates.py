"""The selective scan where a row's time steps sum to more than fp32 holds, or to 0 beside a rate
that is no number: rows cut into segments give what whole rows give."""
import numpy as np
import pytest

from oracle import ssm
from tests import _mixer as m

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("saved", [True, False])
def test_states_without_decay_under_endless_steps(saved):
    """A rate of 0 keeps a state whatever the time steps, whose sum over a segment passes fp32
    here; a rate of -1 loses it at once.  All terms are positive and no decay is between 0
    and 1, so a result is off by its additions alone: at most 16 states, 8 tokens and 16 joins of
    2^-24 each, less than 2^-18."""
    import recurrent_state_memory_amd as gdr
    T, C, N = 1000, 64, 16
    rng = np.random.default_rng(11)
    A = np.zeros((C, N), np.float32)
    A[:, 1::2] = -1
    x, dt, gy = (np.zeros((1, T, C), np.float32) for _ in range(3))
    dt[:] = 2e37
    gy[:, -8:] = rng.uniform(0.5, 1, (1, 8, C))
    Bv = rng.uniform(2.0 ** -8, 2.0 ** -7, (1, T, 1, N)).astype(np.float32)
    Cv = rng.uniform(0.5, 1, (1, T, 1, N)).astype(np.float32)
    h0, dh = rng.uniform(0.5, 1, (2, 1, C, N)).astype(np.float32)
    t = [m.dev(v) for v in (x, dt, A, Bv, Cv)]
    y, h, ck = gdr.gdr_ssm_fwd(*t, h0=m.dev(h0), return_ckpt=True)
    g = gdr.gdr_ssm_bwd(m.dev(gy), *t, h0=None if saved else m.dev(h0), ckpt=ck if saved else None, grad_h=m.dev(dh))
    y_r, h_r, ck_r = ssm.forward(x, dt, A, Bv, Cv, h0=h0)
    g_r = ssm.backward(gy, x, dt, A, Bv, Cv, h0=h0, dh=dh)
    for k, a, r in [("y", y, y_r), ("h", h, h_r), ("ckpt", ck, ck_r),
                    *((k, g[k], g_r["d" + k]) for k in ("x", "B", "C", "h0")), ("dt", g["dt"], g_r["ddt"])]:
        np.testing.assert_allclose(m.host(a), r, rtol=2.0 ** -18, atol=0, err_msg=k)


@pytest.mark.parametrize("N", [4, 16, 20])
def test_empty_rows_pass_states_on(N):
    """A row without tokens passes every state and every adjoint on as it is, whatever the
    rates, in a long batch (whose rows are cut into segments) as in a short one."""
    import torch
    import recurrent_state_memory_amd as gdr
    for T in (40, 700):
        d = m.ssm_inputs(2, T, 70, N, 1, "f32", 21)
        d["A"][3], d["A"][69], d["A"][40, 1], d["A"][41, 2] = np.nan, -np.inf, np.inf, -3e38
        t = [m.dev(d[k]) for k in ("x", "dt", "A", "Bv", "Cv")]
        kw = dict(dt_bias=m.dev(d["dt_bias"]), lens=m.as_int32([0, T]))
        h0, dh = m.dev(d["h0"]), m.dev(d["dh"])
        y, h, ck = gdr.gdr_ssm_fwd(*t, h0=h0, return_ckpt=True, **kw)
        assert torch.equal(h[0], h0[0]) and not bool(y[0].any())
        assert all(torch.equal(c, h0[0].t()) for c in ck[0])
        for start in (dict(h0=h0), dict(ckpt=ck)):
            g = gdr.gdr_ssm_bwd(m.dev(d["dy"]), *t, grad_h=dh, **start, **kw)
            assert torch.equal(g["h0"][0], dh[0])
            assert not any(bool(g[k][0].any()) for k in ("x", "dt", "B", "C"))
