"""Parity of the channelwise recurrence (gdr_scan_fwd, gdr_scan_bwd,
gdr_scan_step) with the fp64 oracle, element by element, within bounds that count
the roundings (tests/_chan.py)."""
import numpy as np
import pytest

from _chan import E, check, dev, gate_bounds, half_step, host, scan_error, scan_inputs
from oracle import ckpt8, scan

pytestmark = pytest.mark.gpu

KINDS = ["alpha", "decay", "gate", "norm", "gate+norm"]


def call_fwd(d, io, **kw):
    import recurrent_state_memory_amd as gdr
    k = d["kw"]
    if "alpha" in k:
        return gdr.gdr_scan_fwd(dev(d["x"], io), dev(k["alpha"]), **kw)
    return gdr.gdr_scan_fwd_gated(dev(d["x"], io), dev(k["d"], io), dev(k["A"]), gate_x=dev(k.get("g"), io),
                                  normalise=k["normalise"], **kw)


def call_bwd(d, io, x=None, **kw):
    import recurrent_state_memory_amd as gdr
    k = d["kw"]
    x = dev(d["x"], io) if x is None else x
    if "alpha" in k:
        return gdr.gdr_scan_bwd(x, dev(k["alpha"]), dev(d["dy"], io), **kw)
    return gdr.gdr_scan_bwd_gated(x, dev(k["d"], io), dev(k["A"]), dev(d["dy"], io), gate_x=dev(k.get("g"), io),
                                  normalise=k["normalise"], **kw)


def check_fwd(d, io, h0, what):
    import torch
    y, h, ck = call_fwd(d, io, h0=dev(h0), return_ckpt=True)
    torch.cuda.synchronize()
    yr, hr, cr = scan.forward(d["x"], h0=h0, **d["kw"])
    q = scan.gates(**d["kw"])
    ra, rb = gate_bounds(q, d["kw"].get("g"))
    start = np.zeros_like(hr) if h0 is None else h0.astype(np.float64)
    after, last, before = scan_error(q["a"], q["b"] * d["x"], ra, rb + 1, start)
    check(what + " y", y, yr, after + half_step(io) * np.abs(yr))
    check(what + " h", h, hr, last)
    check(what + " ckpt", ck, cr, before[:, ::32])


def check_bwd(d, io, h0, dh, what, x8=False, ck=False):
    import torch
    B, T, C = d["x"].shape
    x, xin = d["x"], None
    ckpt = scan.forward(d["x"], h0=h0, **d["kw"])[2].astype(np.float32) if ck else None
    if x8:
        code, exp = ckpt8.pack(x.reshape(B * T, C))
        x = ckpt8.value(code, exp).reshape(B, T, C)
        xin = (torch.from_numpy(code.reshape(B, T, C)).cuda().view(torch.float8_e4m3fn),
               torch.from_numpy(exp.reshape(B, T, -1)).cuda())
    g = call_bwd(d, io, x=xin, grad_h=dev(dh), **(dict(ckpt=dev(ckpt)) if ck else dict(h0=dev(h0))))
    torch.cuda.synchronize()
    r = scan.backward(x, d["dy"], dh, h0=h0, ckpt=ckpt, **d["kw"])
    q, G, prev = r["q"], r["G"], r["prev"]
    a, b, v = q["a"], q["b"], q["b"] * x
    ra, rb = gate_bounds(q, d["kw"].get("g"))
    if ck:                      # each block starts from an exact state
        Np = np.zeros_like(x)
        for j in range(0, T, 32):
            s = np.s_[:, j:j + 32]
            at = [np.broadcast_to(z, x.shape)[s] for z in (ra, rb + 1)]
            Np[s] = scan_error(a[s], v[s], *at, ckpt[:, j // 32].astype(np.float64))[2]
    else:
        start = np.zeros((B, C)) if h0 is None else h0.astype(np.float64)
        Np = scan_error(a, v, ra, rb + 1, start)[2]
    # G runs backwards with the decay of the token behind it
    end = np.zeros((B, C)) if dh is None else dh.astype(np.float64)
    af = np.concatenate([np.ones((B, 1, C)), a[:, :0:-1]], 1)
    raf = np.broadcast_to(ra, x.shape)
    raf = np.concatenate([np.zeros((B, 1, C)), raf[:, :0:-1]], 1)
    NG, _, _ = scan_error(af, d["dy"][:, ::-1].astype(np.float64), raf, 0.0, end)
    NG = NG[:, ::-1]
    hs, Ga = half_step(io), np.abs(G)
    check(what + " dx", g["x"], r["dx"], NG * b + Ga * b * (rb + 2) * E + hs * np.abs(r["dx"]))
    if "h0" in g:
        check(what + " dh0", g["h0"], r["dh0"], (a * NG + a * Ga * (ra + 2) * E)[:, 0])
    if "alpha" in d["kw"]:
        check(what + " dalpha", g["alpha"], r["dalpha"], NG * np.abs(prev) + Ga * Np + 2 * E * np.abs(r["dalpha"]))
        return
    if "g" in d["kw"]:
        gs = np.abs(v) * (1 - q["s"])
        # 1 - s: s is off by 2 (|g| + 1) + 4 of itself
        es = np.abs(v) * q["s"] * (2 * np.abs(d["kw"]["g"]) + 7) * E
        check(what + " dg", g["gate_x"], r["dg"], NG * gs + Ga * (gs * (rb + 5) * E + es) + hs * np.abs(r["dg"]))
    inner, ei = np.abs(prev), Np
    if q["m"] is not None:
        w = np.where(q["m"] > 0, np.abs(v) * a / np.where(q["m"] > 0, q["m"], 1), 0.0)
        inner = inner + w
        ei = ei + w * (rb + ra + q["rm"] + 6) * E
    edu = NG * a * inner + Ga * a * ((ra + 4) * E * inner + ei)
    A = d["kw"]["A"].astype(np.float64)
    check(what + " dd", g["decay_x"], r["dd"],
          edu * A * q["sig"] + np.abs(r["dd"]) * (12 * E + hs + q["neg"] * E))
    # the sum over tokens: at most 64 + (B T) / 32 additions behind any value; the
    # softplus' own error beside them
    k = min(B * T, 64 + B * T // 32) + 10 + q["neg"]
    check(what + " dA", g["decay_a"], r["dA"], (edu * q["sp"] + np.abs(r["du"] * q["sp"]) * k * E).sum((0, 1)))


# lengths around the 32-token blocks and the kernels' tiles, widths that do and do
# not divide by 4 or fill 64 channels
SHAPES = [(1, 1, 1), (2, 1, 64), (1, 31, 4), (3, 33, 66), (2, 64, 128), (1, 127, 63), (2, 257, 68), (1, 700, 5),
          (2, 513, 132)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scan_fwd(shape, kind, io):
    B, T, C = shape
    d = scan_inputs((B, T), C, io, kind, seed=T * 7 + C, reset=T % 2 == 1)
    check_fwd(d, io, d["h"] if C % 2 == 0 else None, f"fwd {kind}/{io}/{shape}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scan_bwd(shape, kind, io):
    B, T, C = shape
    d = scan_inputs((B, T), C, io, kind, seed=T * 11 + C, reset=T % 2 == 1)
    full = C % 2 == 0
    for ck in (False, True):
        check_bwd(d, io, d["h"] if full else None, d["dh"] if full else None, f"bwd {kind}/{io}/{shape}/ckpt={ck}",
                  ck=ck)


@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("kind", ["alpha", "gate+norm"])
@pytest.mark.parametrize("shape", [(2, 45, 63), (1, 290, 132), (2, 33, 260)], ids=str)
def test_scan_bwd_from_8_bits(shape, kind, ck):
    """x kept in 8 bits: the gradients are those of the values that the codes stand for."""
    B, T, C = shape
    for io in ("bf16", "f32"):
        d = scan_inputs((B, T), C, io, kind, seed=T + C)
        check_bwd(d, io, d["h"], d["dh"], f"bwd8 {kind}/{io}/{shape}/ckpt={ck}", x8=True, ck=ck)


def test_scan_long():
    """Many tiles of one chain: 20000 tokens, slow and fast channels, resets."""
    d = scan_inputs((1, 20011), 8, "f32", "alpha", seed=3, reset=True)
    check_fwd(d, "f32", d["h"], "long")
    d = scan_inputs((1, 9001), 6, "bf16", "gate+norm", seed=4)
    check_fwd(d, "bf16", d["h"], "long gated")
    check_bwd(d, "bf16", d["h"], d["dh"], "long gated bwd")


@pytest.mark.parametrize("T", [255, 256, 257, 1100, 2049, 5000])
@pytest.mark.parametrize("kind", ["alpha", "norm"])
def test_scan_remembers(kind, T):
    """Channels that keep their start state (and the last gradient) over the whole
    sequence, beside ones that forget within some hundred tokens: a state lost or
    taken twice anywhere along the tiles shows at its full size."""
    B, C = 2, 70
    d = scan_inputs((B, T), C, "f32", kind, seed=T)
    A = np.exp(np.linspace(np.log(1e-7), np.log(0.05), C)).astype(np.float32)
    if kind == "alpha":
        d["kw"]["alpha"] = np.exp(-A * np.logaddexp(0, d["x"][:, ::-1])).astype(np.float32)
    else:
        d["kw"]["A"] = A
    d["x"] = d["x"] * np.float32(0.01)
    d["dy"] = d["dy"] * np.float32(0.01)
    check_fwd(d, "f32", d["h"], f"remembers {kind}/{T}")
    for ck in (False, True):
        check_bwd(d, "f32", d["h"], d["dh"], f"remembers {kind}/{T}/ckpt={ck}", ck=ck)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,C", [(1, 1), (1, 2048), (7, 66), (256, 64), (3, 1001)])
def test_scan_step(N, C, kind, io):
    import torch
    import recurrent_state_memory_amd as gdr
    d = scan_inputs((N,), C, io, kind, seed=N + C)
    k = d["kw"]
    want = scan.step(d["h"], d["x"], **k)
    q = scan.gates(**k)
    ra, rb = gate_bounds(q, k.get("g"))
    tol = q["a"] * np.abs(d["h"]) * (ra + 2) * E + np.abs(q["b"] * d["x"]) * (rb + 2) * E + E * np.abs(want)
    for inplace in (True, False):
        h = dev(d["h"])
        out = None if inplace else torch.full_like(h, float("nan"))
        if "alpha" in k:
            y = gdr.gdr_scan_step(h, dev(d["x"], io), dev(k["alpha"]), h_out=out)
        else:
            y = gdr.gdr_scan_step_gated(h, dev(d["x"], io), dev(k["d"], io), dev(k["A"]), gate_x=dev(k.get("g"), io),
                                        normalise=k["normalise"], h_out=out)
        torch.cuda.synchronize()
        check(f"step {kind}/{io} h", h if inplace else out, want, tol)
        check(f"step {kind}/{io} y", y, want, tol + half_step(io) * np.abs(want))
        if not inplace:
            assert torch.equal(h, dev(d["h"]))


def test_steps_continue_the_scan():
    """A prefix by the scan, then single tokens on its final state: the scan's own outputs."""
    import torch
    import recurrent_state_memory_amd as gdr
    d = scan_inputs((3, 40), 132, "f32", "gate+norm", seed=8)
    y, _, _ = call_fwd(d, "f32", h0=dev(d["h"]))
    cut = dict(d, x=d["x"][:, :37], kw={k: (v[:, :37] if getattr(v, "ndim", 0) == 3 else v) for k, v in d["kw"].items()})
    _, h, _ = call_fwd(cut, "f32", h0=dev(d["h"]))
    for t in range(37, 40):
        k = d["kw"]
        yt = gdr.gdr_scan_step_gated(h, dev(d["x"][:, t]), dev(k["d"][:, t]), dev(k["A"]), gate_x=dev(k["g"][:, t]))
        # the same token from states that differ by a few roundings
        assert torch.allclose(yt, y[:, t], rtol=0, atol=64 * E * float(y.abs().max()))


def test_scan_h_out_may_be_h0():
    import torch
    d = scan_inputs((2, 300), 64, "bf16", "alpha", seed=9)
    h0 = dev(d["h"])
    _, h, _ = call_fwd(d, "bf16", h0=h0.clone())
    _, h2, _ = call_fwd(d, "bf16", h0=h0, h_out=h0)
    assert h2 is h0 and torch.equal(h, h2)


def test_scan_saturated_gates():
    """Pre-activations at the ends of their range: no NaN where the formula has none."""
    import torch
    import recurrent_state_memory_amd as gdr
    d = np.array([-np.inf, -200.0, -90.0, -20.0, 0.0, 20.0, 200.0, 3e38], np.float32).reshape(1, 8, 1).repeat(4, 2)
    g = np.array([3e38, -3e38, 200.0, -200.0], np.float32).reshape(1, 1, 4).repeat(8, 1)
    x, A = np.ones((1, 8, 4), np.float32), np.full(4, 0.5, np.float32)
    y, h, _ = gdr.gdr_scan_fwd_gated(dev(x), dev(d), dev(A), gate_x=dev(g), h0=dev(np.ones((1, 4))))
    yr = scan.forward(x, h0=np.ones((1, 4)), d=d, A=A, g=g, normalise=True)[0]
    assert np.abs(host(y) - yr).max() <= 1e-5
    gr = gdr.gdr_scan_bwd_gated(dev(x), dev(d), dev(A), dev(x), gate_x=dev(g), h0=dev(np.ones((1, 4))))
    for n, t in gr.items():
        assert torch.isfinite(t).all(), n
    # an infinite pre-activation is the reset that a very large one is, gradients included
    d[0, 7], d[0, 3] = np.inf, 3e38
    dm = np.where(np.isinf(d) & (d > 0), np.float32(3e38), d)
    outs = []
    for dd in (d, dm):
        y, h, ck = gdr.gdr_scan_fwd_gated(dev(x), dev(dd), dev(A), gate_x=dev(g), h0=dev(np.ones((1, 4))), return_ckpt=True)
        g2 = gdr.gdr_scan_bwd_gated(dev(x), dev(dd), dev(A), dev(x), gate_x=dev(g), ckpt=ck)
        outs.append([y, h, *g2.values()])
    assert all(torch.isfinite(a).all() and torch.equal(a, b) for a, b in zip(*outs))


def test_scan_padded_batch():
    """Padding (decay_x = -Inf with normalise) behind rows of different lengths: the
    final states and every gradient are those of the rows alone, and the padding's are 0."""
    import torch
    d = scan_inputs((3, 300), 70, "bf16", "gate+norm", seed=70)
    lens = (300, 129, 37)
    for b, n in enumerate(lens):
        d["kw"]["d"][b, n:] = -np.inf
        d["dy"][b, n:] = 0.0
    _, h, _ = call_fwd(d, "bf16", h0=dev(d["h"]))
    g = call_bwd(d, "bf16", h0=dev(d["h"]), grad_h=dev(d["dh"]))
    for b, n in enumerate(lens):
        one = dict(x=d["x"][b:b + 1, :n], dy=d["dy"][b:b + 1, :n], kw=dict(d["kw"], d=d["kw"]["d"][b:b + 1, :n], g=d["kw"]["g"][b:b + 1, :n]))
        _, h1, _ = call_fwd(one, "bf16", h0=dev(d["h"][b:b + 1]))
        g1 = call_bwd(one, "bf16", h0=dev(d["h"][b:b + 1]), grad_h=dev(d["dh"][b:b + 1]))
        assert torch.equal(h[b], h1[0]) and torch.equal(g["h0"][b], g1["h0"][0])
        for k in ("x", "decay_x", "gate_x"):
            assert torch.equal(g[k][b, :n], g1[k][0]) and (g[k][b, n:] == 0).all(), (b, k)


def test_scan_nan_stays_in_its_channel():
    import torch
    d = scan_inputs((2, 100), 70, "f32", "gate+norm", seed=10)
    clean = call_fwd(d, "f32", h0=dev(d["h"]))[0]
    d["x"][1, 50, 33] = np.nan
    y = call_fwd(d, "f32", h0=dev(d["h"]))[0]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 50:, 33] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("T", [100, 130])
def test_scan_nan_in_the_last_token(T):
    """A NaN that reaches the state with the last token alone leaves every gradient
    that does not read it finite (the tile's rows behind T included)."""
    import torch
    d = scan_inputs((1, T), 64, "f32", "decay", seed=T)
    clean = call_bwd(d, "f32", h0=dev(d["h"]), grad_h=dev(d["dh"]))
    d["x"][0, T - 1, 7] = np.nan
    g = call_bwd(d, "f32", h0=dev(d["h"]), grad_h=dev(d["dh"]))
    assert all(torch.equal(g[k], clean[k]) for k in clean)


def test_scan_writes_only_its_outputs():
    """Outputs inside larger buffers: the bytes around them stay as they were; the
    results are the same at every alignment."""
    import torch
    for C, off in ((64, 64), (64, 1), (33, 3)):
        d = scan_inputs((2, 77), C, "bf16", "gate+norm", seed=C)
        n = 2 * 77 * C
        buf = torch.full((n + 200,), 7.0, dtype=torch.bfloat16, device="cuda")
        hb = torch.full((2 * C + 200,), 7.0, device="cuda")
        cb = torch.full((2 * 3 * C + 200,), 7.0, device="cuda")
        y, h, ck = (b[off:off + k].view(s) for b, k, s in ((buf, n, (2, 77, C)), (hb, 2 * C, (2, C)),
                                                           (cb, 6 * C, (2, 3, C))))
        call_fwd(d, "bf16", h0=dev(d["h"]), y=y, h_out=h, ckpt=ck)
        ref = call_fwd(d, "bf16", h0=dev(d["h"]), return_ckpt=True)
        torch.cuda.synchronize()
        for got, want in zip((y, h, ck), ref):
            assert torch.equal(got, want)
        for b, k in ((buf, n), (hb, 2 * C), (cb, 6 * C)):
            assert (b[:off] == 7).all() and (b[off + k:] == 7).all()


def test_scan_repeats_bit_for_bit():
    import torch
    d = scan_inputs((3, 1500), 200, "bf16", "gate+norm", seed=12)
    first = call_fwd(d, "bf16", h0=dev(d["h"]), return_ckpt=True)
    fb = call_bwd(d, "bf16", h0=dev(d["h"]), grad_h=dev(d["dh"]))
    for _ in range(3):
        again = call_fwd(d, "bf16", h0=dev(d["h"]), return_ckpt=True)
        ab = call_bwd(d, "bf16", h0=dev(d["h"]), grad_h=dev(d["dh"]))
        assert all(torch.equal(x, y) for x, y in zip(first, again))
        assert all(torch.equal(fb[k], ab[k]) for k in fb)


def test_scan_given_workspaces():
    """Workspaces that held something else before, used again by a smaller and a larger call."""
    import torch
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    for T, C in ((1000, 130), (300, 64), (3000, 260)):
        d = scan_inputs((2, T), C, "bf16", "gate+norm", seed=T)
        ref, rg = call_fwd(d, "bf16", h0=dev(d["h"])), call_bwd(d, "bf16", h0=dev(d["h"]))
        got = call_fwd(d, "bf16", h0=dev(d["h"]), workspace=ws)
        gg = call_bwd(d, "bf16", h0=dev(d["h"]), workspace=ws)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
        assert all(torch.equal(rg[k], gg[k]) for k in rg)
    with pytest.raises(ValueError, match="workspace"):
        call_fwd(d, "bf16", workspace=ws[:64])


def test_scan_two_graphs_of_one_process():
    """Two captured calls replayed in turn and again: neither finds the other's words."""
    import torch
    import recurrent_state_memory_amd as gdr
    ds = [scan_inputs((2, 700 + 600 * i), 96, "f32", "alpha", seed=60 + i) for i in range(2)]
    ins = [(dev(d["x"]), dev(d["kw"]["alpha"]), dev(d["h"])) for d in ds]
    want = [gdr.gdr_scan_fwd(x, a, h0=h) for x, a, h in ins]
    graphs, outs = [], []
    for x, a, h in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gdr.gdr_scan_fwd(x, a, h0=h))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        for t in outs[i][:2]:
            t.fill_(7)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
        gdr.gdr_scan_fwd(*ins[i][:2])


def test_scan_streams_and_graph():
    """Two streams at once, then forward and backward captured and replayed with new
    inputs and eager calls in between."""
    import torch
    import recurrent_state_memory_amd as gdr
    ds = [scan_inputs((2, 900), 128, "bf16", "gate+norm", seed=20 + i) for i in range(2)]
    want = [call_fwd(d, "bf16", h0=dev(d["h"])) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    ins = [{k: dev(v, None if k == "A" else "bf16") for k, v in d["kw"].items() if k != "normalise"} for d in ds]
    xs, hs = [dev(d["x"], "bf16") for d in ds], [dev(d["h"]) for d in ds]
    torch.cuda.synchronize()
    outs = [[] for _ in ds]
    for _ in range(4):
        for i in range(2):
            outs[i].append(gdr.gdr_scan_fwd_gated(xs[i], ins[i]["d"], ins[i]["A"], gate_x=ins[i]["g"], h0=hs[i],
                                                  stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y, h, _ in outs[i]:
            assert torch.equal(y, want[i][0]) and torch.equal(h, want[i][1])

    x, h, dy = xs[0].clone(), hs[0].clone(), dev(ds[0]["dy"], "bf16")

    def both():
        y, ho, ck = gdr.gdr_scan_fwd_gated(x, ins[0]["d"], ins[0]["A"], gate_x=ins[0]["g"], h0=h, return_ckpt=True)
        return y, gdr.gdr_scan_bwd_gated(x, ins[0]["d"], ins[0]["A"], dy, gate_x=ins[0]["g"], ckpt=ck)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gg = both()
    for i in (1, 0, 1):
        x.copy_(xs[i])
        h.copy_(hs[i])
        graph.replay()
        torch.cuda.synchronize()
        ey, eg = both()
        torch.cuda.synchronize()
        assert torch.equal(gy, ey) and all(torch.equal(gg[k], eg[k]) for k in eg)
