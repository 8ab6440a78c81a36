"""The 8-bit checkpoints against the oracle that enumerates the codes: packing and
unpacking are exact, so every byte and every value has to agree.  And a run of
the channelwise operators together, as a layer uses them."""
import numpy as np
import pytest

from _chan import check, dev, host
from oracle import ckpt8, norm, scan
from synth.gen import bf16_round

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (2, 3), (5, 127), (3, 128), (7, 129), (2, 250), (4, 256), (3, 1000), (2, 2048), (33, 64), (1, 5003)]


def values(R, D, io, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, D)) * 10.0 ** rng.uniform(-6, 6, (R, 1))
    x[rng.uniform(size=(R, D)) < 0.1] *= 1e-3
    x[rng.uniform(size=(R, D)) < 0.05] = 0.0
    x = x.astype(np.float32)
    return bf16_round(x) if io == "bf16" else x


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", SHAPES)
def test_ckpt8_round_trip(R, D, io):
    import torch
    import recurrent_state_memory_amd as gdr
    x = values(R, D, io, R + D)
    code, exp = gdr.gdr_ckpt8_pack(dev(x, io))
    cr, er = ckpt8.pack(x)
    assert np.array_equal(exp.cpu().numpy(), er)
    assert np.array_equal(code.view(torch.uint8).cpu().numpy(), cr)
    want = ckpt8.value(cr, er)
    for dt in (torch.bfloat16, torch.float32):
        got = gdr.gdr_ckpt8_unpack(code, exp, dtype=dt)
        assert got.dtype == dt and np.array_equal(host(got), want)   # 4 significant bits: exact in both
    assert np.abs(want - x).max() <= 2.0 ** -4 * np.abs(x).max()


def test_ckpt8_every_code_and_ties():
    """All 256 codes to numbers; the midpoints between neighbours to the even code."""
    import torch
    import recurrent_state_memory_amd as gdr
    c = np.arange(256, dtype=np.uint8).reshape(2, 128)
    for E in (1, 100, 127, 200):
        e = np.full((2, 1), E, np.uint8)
        got = host(gdr.gdr_ckpt8_unpack(torch.from_numpy(c).cuda().view(torch.float8_e4m3fn),
                                        torch.from_numpy(e).cuda(), dtype=torch.float32))
        want = ckpt8.value(c, e)
        assert np.array_equal(got, want, equal_nan=True)
    mid = (ckpt8.MAGNITUDE[:-1] + ckpt8.MAGNITUDE[1:]) / 2
    x = np.concatenate([mid, [448.0, 0.0]]).astype(np.float32).reshape(1, 128)
    for s in (1.0, -1.0):
        code, exp = gdr.gdr_ckpt8_pack(dev(s * x))
        cr, er = ckpt8.pack(s * x)
        assert np.array_equal(code.view(torch.uint8).cpu().numpy() & 127, cr & 127) and np.array_equal(exp.cpu().numpy(), er)


def test_ckpt8_largest_of_a_group_and_ends_of_the_range():
    """Maxima on both sides of 448 times a power of two, denormals, the largest float, NaN and Inf."""
    import torch
    import recurrent_state_memory_amd as gdr
    rows = []
    for top in (448.0, np.nextafter(np.float32(448), np.float32(1e9)), 447.9, 1.0, 1.75, 1.7500001, 3.4028235e38,
                2.0 ** -126, 1e-40, 1e-45, 2.0 ** -118 * 1.75, 2.0 ** -118):
        r = np.zeros(130, np.float32)
        r[7], r[9], r[129] = top, -top / 3, top
        rows.append(r)
    r = np.zeros(130, np.float32)
    r[[0, 1, 2, 3]] = np.nan, np.inf, -np.inf, 5.0
    rows += [r, np.full(130, np.inf, np.float32)]
    x = np.stack(rows)
    code, exp = gdr.gdr_ckpt8_pack(dev(x))
    cr, er = ckpt8.pack(x)
    assert np.array_equal(exp.cpu().numpy(), er)
    got, want = code.view(torch.uint8).cpu().numpy(), cr
    nan = (want & 127) == 127
    assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan])
    v = host(gdr.gdr_ckpt8_unpack(code, exp, dtype=torch.float32))
    # the largest float rounds up to 2^128, which fp32 holds as Inf
    with np.errstate(over="ignore"):
        want = ckpt8.value(cr, er).astype(np.float32)
    assert np.isinf(want[6, 129]) and np.array_equal(v, want.astype(np.float64), equal_nan=True)


def test_ckpt8_large_and_its_surroundings():
    """Many rows, leading dimensions, an output in a larger buffer at an odd offset."""
    import torch
    import recurrent_state_memory_amd as gdr
    x = values(6000, 200, "bf16", 5)
    code, exp = gdr.gdr_ckpt8_pack(dev(x, "bf16").view(20, 300, 200))
    assert code.shape == (20, 300, 200) and exp.shape == (20, 300, 2)
    buf = torch.full((6000 * 200 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[5:5 + 6000 * 200].view(20, 300, 200)
    gdr.gdr_ckpt8_unpack(code, exp, x=out)
    assert (buf[:5] == 7).all() and (buf[5 + 6000 * 200:] == 7).all()
    xd = x.astype(np.float64).reshape(6000, 200)
    top = np.stack([np.abs(xd[:, :128]).max(1), np.abs(xd[:, 128:]).max(1)], 1)
    scale = 2.0 ** (exp.cpu().numpy().reshape(6000, 2).astype(np.float64) - 127)
    assert np.all(top <= 448 * scale) and np.all((top > 224 * scale) | (scale == 2.0 ** -126))
    err = np.abs(host(out).reshape(6000, 200) - xd)
    per = np.repeat(scale, 128, 1)[:, :200]
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(xd), 2.0 ** -10 * per))


def test_layer_run():
    """A pre-norm recurrent layer's training step from the operators together: norm
    (keeping its input in 8 bits), projections, gated scan (keeping its states, and
    its input in 8 bits), and back.  The gradients against the same step in fp64 on
    the values that the kept codes stand for."""
    import torch
    import recurrent_state_memory_amd as gdr
    rng = np.random.default_rng(17)
    B, T, D = 2, 130, 256
    f64 = np.float64
    x = bf16_round(rng.standard_normal((B, T, D)).astype(np.float32))
    w, b = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32), (0.1 * rng.standard_normal(D)).astype(np.float32)
    A = np.exp(rng.uniform(np.log(0.01), 0, D)).astype(np.float32)
    W = [bf16_round((rng.standard_normal((D, D)) / 16).astype(np.float32)) for _ in range(3)]
    dy = bf16_round(rng.standard_normal((B, T, D)).astype(np.float32))
    Wd = [dev(m, "bf16") for m in W]

    n, mean, rstd, kept = gdr.gdr_norm_fwd(dev(x, "bf16"), dev(w), dev(b), return_ckpt8=True)
    u, d, g = (n.view(-1, D) @ m for m in Wd)
    u, d, g = (t.view(B, T, D) for t in (u, d, g))
    y, _, ck = gdr.gdr_scan_fwd_gated(u, d, dev(A), gate_x=g, return_ckpt=True)
    u8 = gdr.gdr_ckpt8_pack(u)
    gr = gdr.gdr_scan_bwd_gated(u8, d, dev(A), dev(dy, "bf16"), gate_x=g, ckpt=ck, need_grad_h0=False)
    dn = sum(t.view(-1, D).float() @ m.float().t() for t, m in zip((gr["x"], gr["decay_x"], gr["gate_x"]), Wd))
    dn = dn.view(B, T, D).bfloat16()
    gn = gdr.gdr_norm_bwd(dn, kept, mean, rstd, dev(w))
    torch.cuda.synchronize()

    # each stage in fp64 on the stage's own (rounded) inputs; bounds: one bf16
    # rounding of an output plus 2^-12 of the largest value for fp32 arithmetic
    def near(name, got, want):
        check(name, got, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * np.abs(want).max())
    yn = norm.forward(x, w, b)[0]
    near("norm", n, yn)
    hu, hd, hg = host(u), host(d), host(g)
    near("scan", y, scan.forward(hu, d=hd, A=A, g=hg, normalise=True)[0])
    code, exp = ckpt8.pack(hu.reshape(-1, D))
    hu8 = ckpt8.value(code, exp).reshape(B, T, D)
    r = scan.backward(hu8, dy, ckpt=host(ck), d=hd, A=A, g=hg, normalise=True)
    for k, rk in (("x", "dx"), ("decay_x", "dd"), ("gate_x", "dg"), ("decay_a", "dA")):
        near("scan d" + k, gr[k], r[rk])
    code, exp = ckpt8.pack(x.reshape(-1, D))
    dx, dw, db, _ = norm.backward(host(dn).reshape(-1, D), ckpt8.value(code, exp), host(mean).ravel(),
                                  host(rstd).ravel(), w)
    near("norm dx", gn["x"].view(-1, D), dx)
    near("norm dw", gn["weight"], dw)
    near("norm db", gn["bias"], db)


def test_delta_rule_backward_from_8_bits():
    """q, k and v of the delta rule kept in 8 bits: gdr_chunk_bwd on the unpacked
    values is the backward of exactly those values."""
    import torch
    import recurrent_state_memory_amd as gdr
    from oracle import grad
    from oracle.errors import max_rel_err
    from synth.gen import Workload, generate
    x = generate(Workload("kept", 1, 2, 70, 64, 64, 64, "bf16", "diag", False, 33))
    kept = [gdr.gdr_ckpt8_pack(dev(t, "bf16")) for t in (x.q, x.k, x.v)]
    q, k, v = (gdr.gdr_ckpt8_unpack(*t) for t in kept)
    dO = bf16_round(np.random.default_rng(3).standard_normal(x.v.shape).astype(np.float32))
    g = gdr.gdr_chunk_bwd(q, k, v, dev(x.alpha), dev(x.w), dev(x.beta), dev(dO, "bf16"))
    torch.cuda.synchronize()
    h = [ckpt8.value(*ckpt8.pack(t.reshape(-1, 64))).reshape(t.shape) for t in (x.q, x.k, x.v)]
    assert all(np.array_equal(host(a), b) for a, b in zip((q, k, v), h))
    ref = grad.backward_seq(*h, x.w, x.alpha, x.beta, dO)
    for nm in ("q", "k", "v", "alpha", "beta", "w"):
        assert max_rel_err(g[nm].cpu().numpy(), ref["d" + nm]) <= 2e-2, nm   # the backward tests' bf16 bar
