"""GPU parity of the selective state space scan against the fp64 oracle, element by element."""
import numpy as np
import pytest

from oracle import ssm
from tests import _mixer as m

pytestmark = pytest.mark.gpu

SHAPES = [  # B, T, C, N, G, padded
    (1, 1, 1, 1, 1, False), (2, 1, 70, 16, 1, False), (1, 31, 3, 5, 1, False), (3, 33, 64, 16, 1, True),
    (2, 64, 65, 8, 1, False), (1, 97, 130, 16, 2, False), (4, 50, 12, 3, 4, True), (1, 200, 64, 4, 1, False),
    (2, 70, 40, 32, 1, True), (1, 65, 66, 64, 1, False), (2, 40, 20, 17, 2, True), (1, 33, 9, 63, 3, False),
    (1, 300, 66, 48, 1, True), (2, 130, 30, 40, 1, True), (1, 600, 64, 2, 1, False), (1, 1500, 20, 33, 2, True),
    (1, 1100, 64, 16, 1, False), (2, 700, 10, 8, 1, True), (7, 130, 96, 16, 1, True),
]


def _lens(B, T, padded):
    return [(T, 0, 1, T // 2, T + 9, -1, T - 1)[b % 7] for b in range(B)] if padded else None


def _opts(i):
    """Which of softplus, gate, skip and bias a case has."""
    return dict(softplus=i % 4 != 3, gate=i % 2 == 0, skip=i % 3 != 1)


def _case(B, T, C, N, G, padded, io, i, seed, wild=False):
    o = _opts(i)
    d = m.ssm_inputs(B, T, C, N, G, io, seed, o["softplus"], wild)
    lens = _lens(B, T, padded)
    if not o["skip"]:
        d["D"] = np.zeros(C, np.float32)
    bias = o["softplus"]
    t = {k: m.dev(d[k], io) for k in ("x", "dt", "Bv", "Cv", "z", "dy")}
    if padded:                       # nothing behind a row's end is read
        for b, n in enumerate(lens):
            for k in t:
                t[k][b, max(n, 0):] = float("nan")
    args = (t["x"], t["dt"], m.dev(d["A"]), t["Bv"], t["Cv"])
    kw = dict(D=m.dev(d["D"]) if o["skip"] else None, z=t["z"] if o["gate"] else None,
              dt_bias=m.dev(d["dt_bias"]) if bias else None, softplus=o["softplus"], lens=m.as_int32(lens))
    ref = dict(D=d["D"], z=d["z"] if o["gate"] else None, dt_bias=d["dt_bias"], softplus=o["softplus"], lens=lens)
    return d, t, args, kw, ref, o


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_forward(i, shape, io):
    import recurrent_state_memory_amd as gdr
    d, t, args, kw, ref, o = _case(*shape, io, i, 10 + i)
    y, h, ck = gdr.gdr_ssm_fwd(*args, h0=m.dev(d["h0"]), return_ckpt=True, **kw)
    r = ssm.backward(d["dy"], d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **ref)
    y_r, h_r, ck_r = ssm.forward(d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **ref)
    ey, eh, before = m.ssm_fwd_bounds(d, r["q"], r["h"], r["prev"], y_r, io, o["softplus"], o["gate"], d["h0"])
    m.check("y", y, y_r, ey)
    m.check("h", h, h_r, eh)
    m.check("ckpt", ck, ck_r, np.swapaxes(before[:, ::32], 2, 3))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_backward(i, shape, io):
    import recurrent_state_memory_amd as gdr
    d, t, args, kw, ref, o = _case(*shape, io, i, 40 + i)
    kept = i % 2 == 1
    ck = ckh = None
    if kept:
        ck = gdr.gdr_ssm_fwd(*args, h0=m.dev(d["h0"]), return_ckpt=True, **kw)[2]
        ckh = m.host(ck)
    g = gdr.gdr_ssm_bwd(t["dy"], *args, h0=None if kept else m.dev(d["h0"]), ckpt=ck, grad_h=m.dev(d["dh"]), **kw)
    r = ssm.backward(d["dy"], d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], ckpt=ckh, dh=d["dh"], **ref)
    e = m.ssm_bwd_bounds(d, r, io, o["softplus"], o["gate"], d["h0"], ckh)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", h0="dh0")
    names.update({"D": "dD"} if o["skip"] else {})
    names.update({"z": "dz"} if o["gate"] else {})
    names.update({"dt_bias": "dbias"} if o["softplus"] else {})
    assert set(g) == set(names)
    for k, rk in names.items():
        m.check("d" + k, g[k], r[rk], e[k])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_time_steps_of_any_size(io):
    """Decays from next to 1 down to exactly 0, forward and backward."""
    import recurrent_state_memory_amd as gdr
    d, t, args, kw, ref, o = _case(2, 150, 70, 16, 1, False, io, 0, 77, wild=True)
    y, h, ck = gdr.gdr_ssm_fwd(*args, h0=m.dev(d["h0"]), return_ckpt=True, **kw)
    ckh = m.host(ck)
    r = ssm.backward(d["dy"], d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **ref)
    y_r, h_r, _ = ssm.forward(d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **ref)
    ey, eh, _ = m.ssm_fwd_bounds(d, r["q"], r["h"], r["prev"], y_r, io, True, True, d["h0"])
    m.check("y", y, y_r, ey)
    m.check("h", h, h_r, eh)
    g = gdr.gdr_ssm_bwd(t["dy"], *args, ckpt=ck, grad_h=m.dev(d["dh"]), **kw)
    r = ssm.backward(d["dy"], d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], ckpt=ckh, dh=d["dh"], **ref)
    e = m.ssm_bwd_bounds(d, r, io, True, True, None, ckh)
    for k, rk in dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", h0="dh0", D="dD", z="dz", dt_bias="dbias").items():
        m.check("d" + k, g[k], r[rk], e[k])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,C,N,G", [(1, 1, 1, 1), (1, 2048, 16, 1), (5, 33, 7, 3), (64, 40, 4, 2), (3, 70, 64, 1), (9, 64, 24, 1),
                                     (2, 300, 2, 4)])
def test_step(R, C, N, G, io):
    import torch
    import recurrent_state_memory_amd as gdr
    for i in range(2):
        o = dict(softplus=i == 0, gate=i == 0)
        d = m.ssm_inputs(R, 1, C, N, G, io, C + i, o["softplus"])
        a = [m.dev(d["x"][:, 0], io), m.dev(d["dt"][:, 0], io), m.dev(d["A"]), m.dev(d["Bv"][:, 0], io), m.dev(d["Cv"][:, 0], io)]
        kw = dict(D=m.dev(d["D"]), z=m.dev(d["z"][:, 0], io) if o["gate"] else None, dt_bias=m.dev(d["dt_bias"]),
                  softplus=o["softplus"])
        h = m.dev(d["h0"])
        out = torch.empty_like(h)
        y = gdr.gdr_ssm_step(h, *a, h_out=out, **kw)
        assert torch.equal(h, m.dev(d["h0"]))
        y1 = gdr.gdr_ssm_step(h, *a, **kw)
        assert torch.equal(y, y1) and torch.equal(h, out)
        rk = dict(D=d["D"], z=d["z"] if o["gate"] else None, dt_bias=d["dt_bias"], softplus=o["softplus"])
        r = ssm.backward(d["dy"], d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **rk)
        y_r, h_r, _ = ssm.forward(d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **rk)
        ey, eh, _ = m.ssm_fwd_bounds(d, r["q"], r["h"], r["prev"], y_r, io, o["softplus"], o["gate"], d["h0"])
        m.check("y", y, y_r[:, 0], ey[:, 0])
        m.check("h", h, h_r, eh)


def test_optional_arguments():
    """Absent inputs count as zeros; outputs may be given, the state overwritten in place."""
    import torch
    import recurrent_state_memory_amd as gdr
    d, t, args, kw, _, _ = _case(2, 75, 40, 16, 1, False, "bf16", 0, 5)
    zc, zh = torch.zeros(40, device="cuda"), torch.zeros(2, 40, 16, device="cuda")
    y, h, ck = gdr.gdr_ssm_fwd(*args)
    y0, h0, ck0 = gdr.gdr_ssm_fwd(*args, D=zc, dt_bias=zc, h0=zh, return_ckpt=True)
    assert ck is None and torch.equal(y, y0) and torch.equal(h, h0)
    assert gdr.gdr_ssm_fwd(*args, return_state=False)[1] is None
    g = gdr.gdr_ssm_bwd(t["dy"], *args, need_grad_h0=False)
    g0 = gdr.gdr_ssm_bwd(t["dy"], *args, D=zc, dt_bias=zc, grad_h=zh, ckpt=ck0)
    assert set(g) == {"x", "dt", "A", "B", "C"}
    assert all(torch.equal(g[k], g0[k]) for k in g)
    hin = m.dev(d["h0"])
    y1, h1, _ = gdr.gdr_ssm_fwd(*args, h0=hin, **kw)
    out, cko = torch.empty_like(y), torch.empty_like(ck0)
    r = gdr.gdr_ssm_fwd(*args, h0=hin, h_out=hin, y=out, ckpt=cko, **kw)
    assert r[0] is out and r[1] is hin and r[2] is cko and torch.equal(out, y1) and torch.equal(hin, h1)


def test_long_rows_in_place():
    """Few channels over many tokens, where segments of a row are worked on side by side:
    the state may still be overwritten in place, and the results are those of pieces."""
    import torch
    import recurrent_state_memory_amd as gdr
    d, t, args, kw, _, _ = _case(1, 5000, 64, 16, 1, False, "f32", 0, 6)
    hin = m.dev(d["h0"])
    y, h, ck = gdr.gdr_ssm_fwd(*args, h0=hin, return_ckpt=True, **kw)
    for _ in range(5):
        hx = hin.clone()
        y1, _, _ = gdr.gdr_ssm_fwd(*args, h0=hx, h_out=hx, **kw)
        assert torch.equal(hx, h) and torch.equal(y1, y)
    cut = 2048
    first = [a[:, :cut].contiguous() if a.dim() > 2 else a for a in args]
    last = [a[:, cut:].contiguous() if a.dim() > 2 else a for a in args]
    kz = dict(kw, z=None)
    ya, ha, _ = gdr.gdr_ssm_fwd(*first, h0=hin, **dict(kz, z=kw["z"][:, :cut].contiguous()))
    yb, hb, _ = gdr.gdr_ssm_fwd(*last, h0=ha, **dict(kz, z=kw["z"][:, cut:].contiguous()))
    scale = float(h.abs().max())
    assert float((hb - h).abs().max()) <= 2 ** -14 * scale
    assert float((torch.cat([ya, yb], 1) - y).abs().max()) <= 2 ** -14 * float(y.abs().max())
    g = gdr.gdr_ssm_bwd(t["dy"], *args, ckpt=ck, grad_h=m.dev(d["dh"]), **kw)
    g1 = gdr.gdr_ssm_bwd(t["dy"], *args, h0=hin, grad_h=m.dev(d["dh"]), **kw)
    assert all(torch.equal(g[k], g1[k]) for k in g)


@pytest.mark.parametrize("saved", [True, False])
def test_growing_states_that_are_zero(saved):
    """Over 64 steps of e^2 a factor passes fp32, but a state (an adjoint) of zero stays zero
    however many such steps run side by side.  The inputs lie at one end, the gradients at
    the other; all numbers are positive, so a result's error is that of its factors: 8 steps
    of (|A| d log2(e) + 3) 2^-24 and 16 terms, twice at most: less than 2^-16."""
    import torch
    import recurrent_state_memory_amd as gdr
    T, C, N = 1000, 64, 16
    rng = np.random.default_rng(3)
    x, gy = np.zeros((1, T, C), np.float32), np.zeros((1, T, C), np.float32)
    x[:, -8:], gy[:, :8] = rng.uniform(0.5, 1, (2, 1, 8, C))
    dt, A = np.ones((1, T, C), np.float32), np.full((C, N), 2, np.float32)
    Bv, Cv = rng.uniform(0.5, 1, (2, 1, T, 1, N)).astype(np.float32)
    t = [m.dev(v) for v in (x, dt, A, Bv, Cv)]
    y, h, ck = gdr.gdr_ssm_fwd(*t, softplus=False, return_ckpt=True)
    g = gdr.gdr_ssm_bwd(m.dev(gy), *t, softplus=False, ckpt=ck if saved else None)
    torch.cuda.synchronize()
    y_r, h_r, _ = ssm.forward(x, dt, A, Bv, Cv, softplus=False)
    g_r = ssm.backward(gy, x, dt, A, Bv, Cv, softplus=False)
    for a, r in [(y, y_r), (h, h_r), *((g[k], g_r["d" + k]) for k in ("x", "dt", "A", "B", "C", "h0"))]:
        np.testing.assert_allclose(a.double().cpu().numpy(), r, rtol=2.0 ** -16, atol=0)
