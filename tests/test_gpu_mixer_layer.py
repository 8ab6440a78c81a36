"""The convolution, the selective scan and the gated group norm as a layer uses them: one
after the other, forward and backward, prompt and single tokens, on streams and in graphs."""
import numpy as np
import pytest

from oracle import conv, gnorm, ssm
from tests import _mixer as m

pytestmark = pytest.mark.gpu


def _layer(B, T, C, N, G, H, io, seed):
    """Weights and inputs of a layer: the convolution ahead, a scan, the norm of H heads
    gated by z behind it."""
    d = m.ssm_inputs(B, T, C, N, G, io, seed)
    d.update({k: v for k, v in m.conv_inputs(B, T, C, 4, io, seed + 1).items() if k in ("w", "b", "st")})
    rng = np.random.default_rng(seed + 2)
    d.update(nw=(1 + 0.1 * rng.standard_normal(C)).astype(np.float32), nb=(0.1 * rng.standard_normal(C)).astype(np.float32), H=H)
    t = {k: m.dev(d[k], io if k in ("x", "dt", "Bv", "Cv", "z", "dy", "st") else None) for k in d if k != "H"}
    return d, t


def _forward(t, H, lens=None, state=None, h0=None):
    import recurrent_state_memory_amd as gdr
    u, cs = gdr.gdr_conv_fwd(t["x"], t["w"], t["b"], state=t["st"] if state is None else state, lens=lens)
    s, h, ck = gdr.gdr_ssm_fwd(u, t["dt"], t["A"], t["Bv"], t["Cv"], D=t["D"], dt_bias=t["dt_bias"],
                               h0=t["h0"] if h0 is None else h0, lens=lens, return_ckpt=True)
    y, _, rstd = gdr.gdr_gnorm_fwd(s, H, t["nw"], t["nb"], z=t["z"], silu=True, center=False)
    return dict(u=u, cs=cs, s=s, h=h, ck=ck, y=y, rstd=rstd)


def _backward(t, H, f, lens=None):
    import recurrent_state_memory_amd as gdr
    n = gdr.gdr_gnorm_bwd(t["dy"], f["s"], None, f["rstd"], H, t["nw"], t["nb"], z=t["z"], silu=True)
    s = gdr.gdr_ssm_bwd(n["x"], f["u"], t["dt"], t["A"], t["Bv"], t["Cv"], D=t["D"], dt_bias=t["dt_bias"], ckpt=f["ck"],
                        grad_h=t["dh"], lens=lens)
    c = gdr.gdr_conv_bwd(s["x"], t["x"], t["w"], t["b"], state=t["st"], lens=lens)
    return dict(n=n, s=s, c=c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,N,G,H,lens", [(2, 90, 64, 16, 1, 4, None), (3, 45, 72, 8, 2, 3, [45, 0, 20]),
                                              (1, 700, 128, 16, 1, 2, None)])
def test_training_step(B, T, C, N, G, H, lens, io):
    """Each operator's results against the oracle on what the one before gave."""
    d, t = _layer(B, T, C, N, G, H, io, 5 + T)
    li = m.as_int32(lens)
    f = _forward(t, H, li)
    g = _backward(t, H, f, li)
    y_r, cs_r, u_r = conv.forward(d["x"], d["w"], d["b"], d["st"], lens)
    m.check("conv", f["u"], y_r, m.conv_bounds(d, 4, True, y_r, u_r, io)[1])
    e = dict(d, x=m.host(f["u"]), z=np.zeros_like(d["z"]))
    kw = dict(D=d["D"], dt_bias=d["dt_bias"], lens=lens)
    s_r, h_r, _ = ssm.forward(e["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **kw)
    gn = m.host(g["n"]["x"])
    r0 = ssm.backward(gn, e["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **kw)
    es, eh, _ = m.ssm_fwd_bounds(e, r0["q"], r0["h"], r0["prev"], s_r, io, True, False, d["h0"])
    m.check("scan", f["s"], s_r, es)
    m.check("state", f["h"], h_r, eh)
    s = m.host(f["s"]).reshape(B * T, C)
    z, dy = d["z"].reshape(B * T, C), d["dy"].reshape(B * T, C)
    n_r, mean, rstd, u = gnorm.forward(s, H, d["nw"], d["nb"], z, True, False)
    m.check("norm", f["y"].reshape(B * T, C), n_r,
            m.gnorm_fwd_bounds(s, H, d["nw"], d["nb"], z, True, False, n_r, mean, rstd, u, io)[0])
    # and back
    rh = m.host(f["rstd"]).reshape(B * T, H)
    r = gnorm.backward(dy, s, mean, rh, H, d["nw"], d["nb"], z, True, False)
    ex, ez, ew, eb = m.gnorm_bwd_bounds(dy, s, mean, rh, H, d["nw"], d["nb"], z, True, False, r, io)
    m.check("norm dx", gn.reshape(B * T, C), r["dx"], ex)
    m.check("norm dz", g["n"]["z"].reshape(B * T, C), r["dz"], ez)
    m.check("norm dw", g["n"]["weight"], r["dw"], ew)
    ckh = m.host(f["ck"])
    e["dy"] = gn
    r = ssm.backward(gn, e["x"], d["dt"], d["A"], d["Bv"], d["Cv"], ckpt=ckh, dh=d["dh"], **kw)
    eb = m.ssm_bwd_bounds(e, r, io, True, False, None, ckh)
    for k, rk in dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", h0="dh0", D="dD", dt_bias="dbias").items():
        m.check("scan d" + k, g["s"][k], r[rk], eb[k])
    e = dict(d, dy=m.host(g["s"]["x"]), dst=np.zeros_like(d["st"]))
    r = conv.backward(e["dy"], d["x"], d["w"], d["b"], d["st"], lens, True)
    _, _, uu = conv.forward(d["x"], d["w"], d["b"], d["st"], None, True)
    eu = m.conv_bounds(d, 4, True, uu, uu, io)[0]
    ex, es, ew, eb = m.conv_bwd_bounds(e, r, 4, True, eu, io, T + B + 300)
    m.check("conv dx", g["c"]["x"], r["dx"], ex)
    m.check("conv dw", g["c"]["weight"], r["dw"], ew)


def test_gradients_against_differences():
    """The scan's gradients along a direction against the difference of the oracle's loss."""
    import recurrent_state_memory_amd as gdr
    B, T, C, N, G = 2, 40, 70, 16, 1
    d, t = _layer(B, T, C, N, G, 2, "f32", 9)
    args = (t["x"], t["dt"], t["A"], t["Bv"], t["Cv"])
    g = gdr.gdr_ssm_bwd(t["dy"], *args, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h0=t["h0"], grad_h=t["dh"])
    names = dict(x="x", dt="dt", A="A", Bv="B", Cv="C", D="D", z="z", dt_bias="dt_bias", h0="h0")
    p = {k: d[k].astype(np.float64) for k in names}
    rng = np.random.default_rng(1)
    v = {k: rng.standard_normal(a.shape) for k, a in p.items()}

    def loss(eps):
        q = {k: p[k] + eps * v[k] for k in p}
        y, h, _ = ssm.forward(q["x"], q["dt"], q["A"], q["Bv"], q["Cv"], D=q["D"], z=q["z"], dt_bias=q["dt_bias"], h0=q["h0"])
        return (y * d["dy"]).sum() + (h * d["dh"]).sum()
    eps = 1e-5
    fd = (loss(eps) - loss(-eps)) / (2 * eps)
    r = ssm.backward(d["dy"], d["x"], d["dt"], d["A"], d["Bv"], d["Cv"], D=d["D"], z=d["z"], dt_bias=d["dt_bias"], h0=d["h0"],
                     dh=d["dh"])
    e = m.ssm_bwd_bounds(d, r, "f32", True, True, d["h0"], None)
    got = sum((m.host(g[k]) * v[n]).sum() for n, k in names.items())
    tol = sum((np.broadcast_to(e[k], p[n].shape) * np.abs(v[n])).sum() for n, k in names.items())
    # the difference: its own rounding (2^-52 of the loss' terms over eps) and eps^2 of the third derivative
    terms = (np.abs(d["dy"]) * np.abs(m.host(gdr.gdr_ssm_fwd(*args, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h0=t["h0"])[0]))).sum()
    far = [loss(3 * eps) - loss(-3 * eps), loss(eps) - loss(-eps)]
    third = abs(far[0] / 3 - far[1]) / (2 * eps)              # 8 times eps^2 / 6 of it
    assert abs(got - fd) <= tol + 2.0 ** -40 * terms / eps + third, (got, fd, tol, third)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_tokens(io):
    """A prompt in one call, the tokens behind it one by one: the states and, to rounding,
    the outputs of one call over all of it."""
    import torch
    import recurrent_state_memory_amd as gdr
    B, T, P, C, N, H = 3, 60, 47, 96, 16, 3
    d, t = _layer(B, T, C, N, 1, H, io, 30)
    whole = _forward(t, H)
    cut = {k: v[:, :P].contiguous() if k in ("x", "dt", "Bv", "Cv", "z") else v for k, v in t.items()}
    f = _forward(cut, H)
    cs, h, ys = f["cs"], f["h"], []
    for i in range(P, T):
        one = {k: t[k][:, i].contiguous() for k in ("x", "dt", "Bv", "Cv", "z")}
        u = gdr.gdr_conv_step(cs, one["x"], t["w"], t["b"])
        s = gdr.gdr_ssm_step(h, u, one["dt"], t["A"], one["Bv"], one["Cv"], D=t["D"], dt_bias=t["dt_bias"])
        ys.append(gdr.gdr_gnorm_fwd(s, H, t["nw"], t["nb"], z=one["z"], silu=True, center=False, return_stats=False)[0])
        assert torch.equal(u, whole["u"][:, i])
    assert torch.equal(cs, whole["cs"])
    e = dict(d, x=m.host(whole["u"]), z=np.zeros_like(d["z"]))
    kw = dict(D=d["D"], dt_bias=d["dt_bias"])
    s_r, h_r, _ = ssm.forward(e["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **kw)
    r = ssm.backward(d["dy"], e["x"], d["dt"], d["A"], d["Bv"], d["Cv"], h0=d["h0"], **kw)
    es, eh, _ = m.ssm_fwd_bounds(e, r["q"], r["h"], r["prev"], s_r, io, True, False, d["h0"])
    m.check("state", h, h_r, eh)
    # the norm passes an error of s on as at most rstd |w silu(z)| (1 + sqrt(D) |xh|) of it; both sides' count
    D = C // H
    s2, z2 = s_r[:, P:].reshape(-1, C), d["z"][:, P:].reshape(-1, C)
    y_r, mean, rstd, u = gnorm.forward(s2, H, d["nw"], d["nb"], z2, True, False)
    ey = m.gnorm_fwd_bounds(s2, H, d["nw"], d["nb"], z2, True, False, y_r, mean, rstd, u, io)[0]
    err = es[:, P:].reshape(-1, H, D)
    xh = (s2.reshape(-1, H, D) * rstd[..., None])
    through = (err + np.abs(xh) * np.sqrt((xh ** 2).mean(-1, keepdims=True) * (err ** 2).mean(-1, keepdims=True))) * rstd[..., None]
    # twice: terms of second order in err * rstd
    through = 2 * through.reshape(-1, C) * np.abs(d["nw"] * conv.silu(z2.astype(np.float64))[0])
    m.check("y", torch.stack(ys, 1).reshape(-1, C), y_r, 2 * ey + through)


def test_streams_and_graph():
    """Two streams at once, then the whole step captured and replayed with new inputs and
    eager calls in between; a second graph lives beside the first."""
    import torch
    import recurrent_state_memory_amd as gdr
    H = 4
    layers = [_layer(1, 600 + 40 * i, 64, 16, 1, H, "bf16", 50 + i)[1] for i in range(2)]
    want = [_forward(t, H) for t in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[], []]
    for _ in range(4):
        for i, t in enumerate(layers):
            u, _ = gdr.gdr_conv_fwd(t["x"], t["w"], t["b"], state=t["st"], stream=streams[i])
            s, h, ck = gdr.gdr_ssm_fwd(u, t["dt"], t["A"], t["Bv"], t["Cv"], D=t["D"], dt_bias=t["dt_bias"], h0=t["h0"],
                                       return_ckpt=True, stream=streams[i])
            y, _, _ = gdr.gdr_gnorm_fwd(s, H, t["nw"], t["nb"], z=t["z"], silu=True, center=False, stream=streams[i])
            outs[i].append((u, s, h, ck, y))
    torch.cuda.synchronize()
    for i, f in enumerate(want):
        for o in outs[i]:
            assert all(torch.equal(a, f[k]) for a, k in zip(o, ("u", "s", "h", "ck", "y")))

    def step(t):
        f = _forward(t, H)
        return f, _backward(t, H, f)
    graphs, kept = [], []
    for t in layers:
        step(t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(step(t))
        graphs.append(g)
    for k, i in enumerate((0, 1, 1, 0, 1, 0)):
        t = layers[i]
        t["x"].copy_(t["x"].roll(k + 1, 1))
        t["h0"].mul_(0.5)
        graphs[i].replay()
        torch.cuda.synchronize()
        f, b = step(t)
        torch.cuda.synchronize()
        assert all(torch.equal(kept[i][0][n], f[n]) for n in f)
        assert all(torch.equal(kept[i][1][o][n], b[o][n]) for o in b for n in b[o])


def test_captured_decoding():
    """The single-token steps in place, captured once and replayed: the eager tokens."""
    import torch
    import recurrent_state_memory_amd as gdr
    B, C, N, H = 5, 64, 16, 4
    _, t = _layer(B, 8, C, N, 1, H, "bf16", 70)
    state = [t["st"].clone(), t["h0"].clone()]
    one = {k: t[k][:, 0].contiguous() for k in ("x", "dt", "Bv", "Cv", "z")}

    def token(cs, h, o):
        u = gdr.gdr_conv_step(cs, o["x"], t["w"], t["b"])
        s = gdr.gdr_ssm_step(h, u, o["dt"], t["A"], o["Bv"], o["Cv"], D=t["D"], z=o["z"], dt_bias=t["dt_bias"])
        return gdr.gdr_gnorm_fwd(s, H, t["nw"], t["nb"], z=o["z"], silu=True, center=False)[0]
    token(t["st"].clone(), t["h0"].clone(), one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token(*state, one)
    eager = [t["st"].clone(), t["h0"].clone()]
    state[0].copy_(t["st"]), state[1].copy_(t["h0"])
    for i in range(8):
        for k in one:
            one[k].copy_(t[k][:, i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, token(*eager, {k: t[k][:, i].contiguous() for k in one}))
        assert torch.equal(state[0], eager[0]) and torch.equal(state[1], eager[1])


def test_given_workspaces_and_guards():
    """Workspaces of the size asked for, with anything in them, and outputs in the middle of
    larger buffers: the same results, nothing written outside."""
    import ctypes

    import torch
    import recurrent_state_memory_amd as gdr
    lib = gdr.load_library()
    B, T, C, N, H = 2, 600, 72, 16, 4
    _, t = _layer(B, T, C, N, 1, H, "bf16", 80)
    args = (t["x"], t["dt"], t["A"], t["Bv"], t["Cv"])
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
    io = [a.data_ptr() for a in args]
    tail = (t["D"].data_ptr(), t["z"].data_ptr(), t["dt_bias"].data_ptr())
    fneed = lib.gdr_ssm_fwd_workspace(ctypes.byref(gdr.SsmArgs(B, T, C, N, 1, 1, 1, 0, *io, *tail, None, None, t["dy"].data_ptr())))
    assert fneed > 0
    y, h, ck = gdr.gdr_ssm_fwd(*args, h0=t["h0"], return_ckpt=True, **kw)

    def inside(ref):
        buf = torch.full((ref.numel() + 512,), 3.0, dtype=ref.dtype, device="cuda")
        return buf, buf[256:256 + ref.numel()].view(ref.shape)

    def untouched(buf):
        return bool((buf[:256] == 3).all()) and bool((buf[-256:] == 3).all())
    for fill in (0, 255):
        ws = torch.full((fneed,), fill, dtype=torch.uint8, device="cuda")
        bufs, outs = zip(*(inside(o) for o in (y, h, ck)))
        gdr.gdr_ssm_fwd(*args, h0=t["h0"], y=outs[0], h_out=outs[1], ckpt=outs[2], workspace=ws, **kw)
        assert torch.equal(outs[0], y) and torch.equal(outs[1], h) and torch.equal(outs[2], ck)
        assert all(untouched(b) for b in bufs)
    with pytest.raises(ValueError, match="workspace"):
        gdr.gdr_ssm_fwd(*args, workspace=ws[:-1], **kw)
    u, _, rstd = gdr.gdr_gnorm_fwd(y, H, t["nw"], t["nb"], center=False)
    for fn, call in (("gdr_ssm_bwd", lambda **k: gdr.gdr_ssm_bwd(t["dy"], *args, h0=t["h0"], grad_h=t["dh"], **kw, **k)),
                     ("gdr_conv_bwd", lambda **k: gdr.gdr_conv_bwd(t["dy"], t["x"], t["w"], t["b"], state=t["st"], **k)),
                     ("gdr_gnorm_bwd", lambda **k: gdr.gdr_gnorm_bwd(t["dy"], y, None, rstd, H, t["nw"], t["nb"], **k))):
        ref = call()
        for fill in (0, 255):       # 255: NaN wherever a number is read that was not written
            ws = torch.full((1 << 26,), fill, dtype=torch.uint8, device="cuda")
            g = call(workspace=ws)
            assert all(torch.equal(g[k], ref[k]) for k in ref), (fn, fill)
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=ws[:64])


def test_results_repeat():
    """The same call gives the same bits, whatever ran before."""
    import torch
    _, t = _layer(2, 400, 130, 16, 1, 2, "bf16", 90)
    f0 = _forward(t, 2)
    b0 = _backward(t, 2, f0)
    for _ in range(3):
        torch.randn(1 << 20, device="cuda").sum()
        f = _forward(t, 2)
        b = _backward(t, 2, f)
        assert all(torch.equal(f[k], f0[k]) for k in f) and all(torch.equal(b[o][k], b0[o][k]) for o in b for k in b[o])


def test_nan_and_inf_stay_in_their_channel():
    """A NaN, or an Inf, reaches its own channel from its token on, and nothing else."""
    import torch
    import recurrent_state_memory_amd as gdr
    B, T, C, N = 2, 70, 66, 16
    _, t = _layer(B, T, C, N, 1, 2, "f32", 95)
    args = [t["x"], t["dt"], t["A"], t["Bv"], t["Cv"]]
    kw = dict(D=t["D"], dt_bias=t["dt_bias"])
    y, h, _ = gdr.gdr_ssm_fwd(*args, **kw)
    u, _ = gdr.gdr_conv_fwd(t["x"], t["w"], t["b"])
    for bad in (float("nan"), float("inf")):
        x = t["x"].clone()
        x[1, 40, 65] = bad
        y1, h1, _ = gdr.gdr_ssm_fwd(x, *args[1:], **kw)
        u1, _ = gdr.gdr_conv_fwd(x, t["w"], t["b"])
        hit = torch.zeros_like(x, dtype=torch.bool)
        hit[1, 40:, 65] = True
        assert torch.equal(y1[~hit], y[~hit]) and not bool(torch.isfinite(y1[hit]).any())
        assert torch.equal(h1[0], h[0]) and torch.equal(h1[1, :65], h[1, :65])
        hit[1, 44:, 65] = False
        assert torch.equal(u1[~hit], u[~hit])
