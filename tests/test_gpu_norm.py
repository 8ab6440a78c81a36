"""Parity of the layer norm (gdr_norm_fwd, gdr_norm_bwd) with the fp64 oracle,
element by element, within bounds that count the roundings (tests/_chan.py)."""
import numpy as np
import pytest

from _chan import check, dev, host, norm_bounds, norm_bwd_bounds
from oracle import ckpt8, norm
from synth.gen import bf16_round

pytestmark = pytest.mark.gpu


def inputs(R, D, io, seed, shift=0.0):
    rng = np.random.default_rng(seed)
    cast = bf16_round if io == "bf16" else (lambda z: z.astype(np.float32))
    x = cast((rng.standard_normal((R, D)) * np.exp(rng.uniform(-2, 2, (R, 1))) + shift).astype(np.float32))
    return dict(x=x, dy=cast(rng.standard_normal((R, D)).astype(np.float32)),
                w=rng.standard_normal(D).astype(np.float32), b=rng.standard_normal(D).astype(np.float32))


# widths around the vector, wave and workgroup sizes; row counts around the rows of a group
SHAPES = [(1, 1), (3, 2), (70, 8), (5, 63), (33, 64), (4, 100), (9, 128), (257, 130), (2, 512), (130, 1000), (3, 1024),
          (17, 2048), (2, 2056), (5, 4096), (3, 5003), (2, 8192), (2, 16384), (1, 16392), (2, 40001), (1, 65536)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", SHAPES)
def test_norm_fwd(R, D, io):
    import torch
    import recurrent_state_memory_amd as gdr
    d = inputs(R, D, io, R + D)
    for affine in (True, False):
        w, b = (d["w"], d["b"]) if affine else (None, None)
        y, m, r, kept = gdr.gdr_norm_fwd(dev(d["x"], io), dev(w), dev(b), return_ckpt8=affine)
        torch.cuda.synchronize()
        yr, mr, rr = norm.forward(d["x"], w, b)
        ty, tm, tr = norm_bounds(d["x"].astype(np.float64), w, mr, rr, 1e-5, yr, io)
        what = f"norm fwd {R}x{D}/{io}"
        check(what + " mean", m, mr, tm)
        check(what + " rstd", r, rr, tr)
        check(what + " y", y, yr, ty)
        if affine:
            code, exp = ckpt8.pack(d["x"])
            assert np.array_equal(kept[1].cpu().numpy(), exp)
            assert np.array_equal(kept[0].view(torch.uint8).cpu().numpy(), code)
        else:
            assert kept is None


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", SHAPES + [(3000, 16), (1027, 200)])
def test_norm_bwd(R, D, io, x8):
    import torch
    import recurrent_state_memory_amd as gdr
    d = inputs(R, D, io, R + D + 1)
    _, mean, rstd = (z.astype(np.float32) for z in norm.forward(d["x"]))
    x, xin = d["x"], dev(d["x"], io)
    if x8:
        code, exp = ckpt8.pack(x)
        x = ckpt8.value(code, exp)
        xin = (torch.from_numpy(code).cuda().view(torch.float8_e4m3fn), torch.from_numpy(exp).cuda())
    for affine in (True, False):
        w = d["w"] if affine else None
        g = gdr.gdr_norm_bwd(dev(d["dy"], io), xin, dev(mean), dev(rstd), dev(w), need_grad_weight=affine,
                             need_grad_bias=affine)
        torch.cuda.synchronize()
        dx, dw, db, xh = norm.backward(d["dy"], x, mean, rstd, w)
        tx, tw, tb = norm_bwd_bounds(d["dy"].astype(np.float64), x.astype(np.float64), mean.astype(np.float64),
                                     rstd.astype(np.float64), w, dx, xh, io)
        what = f"norm bwd {R}x{D}/{io}/x8={x8}"
        check(what + " dx", g["x"], dx, tx)
        if affine:
            check(what + " dw", g["weight"], dw, tw)
            check(what + " db", g["bias"], db, tb)
        else:
            assert set(g) == {"x"}


def test_norm_one_column_sum_at_a_time():
    import recurrent_state_memory_amd as gdr
    import torch
    d = inputs(50, 96, "f32", 3)
    _, m, r = (z.astype(np.float32) for z in norm.forward(d["x"]))
    args = (dev(d["dy"]), dev(d["x"]), dev(m), dev(r), dev(d["w"]))
    both = gdr.gdr_norm_bwd(*args)
    w = gdr.gdr_norm_bwd(*args, need_grad_bias=False)
    b = gdr.gdr_norm_bwd(*args, need_grad_weight=False)
    assert set(w) == {"x", "weight"} and set(b) == {"x", "bias"}
    assert torch.equal(both["weight"], w["weight"]) and torch.equal(both["bias"], b["bias"])
    assert torch.equal(both["x"], w["x"]) and torch.equal(both["x"], b["x"])


def test_norm_shifted_and_constant_rows():
    """A mean far from zero against the spread, and rows without any spread."""
    import recurrent_state_memory_amd as gdr
    d = inputs(40, 777, "f32", 4, shift=100.0)
    y, m, r, _ = gdr.gdr_norm_fwd(dev(d["x"]))
    yr, mr, rr = norm.forward(d["x"])
    ty, tm, tr = norm_bounds(d["x"].astype(np.float64), None, mr, rr, 1e-5, yr, "f32")
    check("shifted mean", m, mr, tm)
    check("shifted rstd", r, rr, tr)
    check("shifted y", y, yr, ty)
    x = np.full((3, 100), 2.5, np.float32)
    x[1] = 0.0
    y, m, r, _ = gdr.gdr_norm_fwd(dev(x), dev(d["w"][:100]), dev(d["b"][:100]))
    # a mean off by 1e-6 of the value times 1 / sqrt(eps) = 316
    assert np.abs(host(y) - d["b"][:100]).max() <= 2.5 * 102 * 2.0 ** -24 * 317 * np.abs(d["w"]).max()
    assert np.abs(host(r) - 1e-5 ** -0.5).max() <= 1e-5 ** -0.5 * 1e-4


def test_norm_nan_stays_in_its_row():
    import torch
    import recurrent_state_memory_amd as gdr
    for D in (64, 130, 2048, 20000):
        d = inputs(9, D, "f32", 5)
        clean = gdr.gdr_norm_fwd(dev(d["x"]))[0]
        d["x"][4, D // 2] = np.nan
        y, m, r, kept = gdr.gdr_norm_fwd(dev(d["x"]), return_ckpt8=True)
        keep = torch.arange(9, device="cuda") != 4
        assert torch.isnan(y[4]).all() and torch.equal(y[keep], clean[keep])
        code, exp = ckpt8.pack(d["x"])
        assert np.array_equal(kept[1].cpu().numpy(), exp)
        got = kept[0].float().cpu().numpy()
        assert np.isnan(got[4, D // 2]) and np.isnan(got).sum() == 1
        dx = gdr.gdr_norm_bwd(dev(d["dy"]), dev(d["x"]), m, r)["x"]
        assert torch.isnan(dx[4]).all() and torch.isfinite(dx[keep]).all()


def test_norm_leading_dimensions_and_alignment():
    """Any leading shape; buffers that are aligned to their element alone; the bytes around them stay."""
    import torch
    import recurrent_state_memory_amd as gdr
    d = inputs(24, 256, "bf16", 6)
    ref = gdr.gdr_norm_fwd(dev(d["x"], "bf16"), dev(d["w"]), dev(d["b"]))
    y, m, r, _ = gdr.gdr_norm_fwd(dev(d["x"], "bf16").view(2, 3, 4, 256), dev(d["w"]), dev(d["b"]))
    assert y.shape == (2, 3, 4, 256) and m.shape == (2, 3, 4) and torch.equal(y.view(24, 256), ref[0])
    y1, none, none2, _ = gdr.gdr_norm_fwd(dev(d["x"], "bf16"), dev(d["w"]), dev(d["b"]), return_stats=False)
    assert none is None and none2 is None and torch.equal(y1, ref[0])
    g = gdr.gdr_norm_bwd(dev(d["dy"], "bf16").view(2, 3, 4, 256), dev(d["x"], "bf16").view(2, 3, 4, 256), m, r,
                         dev(d["w"]))
    assert g["x"].shape == (2, 3, 4, 256) and g["weight"].shape == (256,)
    n = 24 * 256
    xb = torch.zeros(n + 9, dtype=torch.bfloat16, device="cuda")
    xb[3:3 + n] = dev(d["x"], "bf16").view(-1)
    yb = torch.full((n + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    y2, m2, r2, _ = gdr.gdr_norm_fwd(xb[3:3 + n].view(24, 256), dev(d["w"]), dev(d["b"]), y=yb[5:5 + n].view(24, 256))
    yr, mr, rr = norm.forward(d["x"], d["w"], d["b"])
    ty, _, _ = norm_bounds(d["x"].astype(np.float64), d["w"], mr, rr, 1e-5, yr, "bf16")
    check("unaligned y", y2, yr, ty)
    assert (yb[:5] == 7).all() and (yb[5 + n:] == 7).all()


def test_norm_of_the_delta_rules_heads():
    """As a layer uses it: gdr_chunk_fwd's output, one norm per head of d_v = 128 channels."""
    import torch
    import recurrent_state_memory_amd as gdr
    from synth.gen import Workload, generate
    x = generate(Workload("heads", 1, 3, 70, 128, 128, 64, "bf16", "diag", False, 31))
    o, _ = gdr.gdr_chunk_fwd(dev(x.q, "bf16"), dev(x.k, "bf16"), dev(x.v, "bf16"), dev(x.alpha), dev(x.w), dev(x.beta))
    y, m, r, _ = gdr.gdr_norm_fwd(o)
    torch.cuda.synchronize()
    on = host(o)
    yr, mr, rr = norm.forward(on)
    ty, _, _ = norm_bounds(on.reshape(-1, 128), None, mr.ravel(), rr.ravel(), 1e-5, yr.reshape(-1, 128), "bf16")
    check("heads y", y, yr, ty.reshape(yr.shape))


def test_norm_one_row_without_leading_dimensions():
    import torch
    import recurrent_state_memory_amd as gdr
    d = inputs(1, 300, "f32", 51)
    x, dy = dev(d["x"]), dev(d["dy"])
    ref = gdr.gdr_norm_fwd(x, return_ckpt8=True)
    y, m, r, kept = gdr.gdr_norm_fwd(x[0], return_ckpt8=True)
    assert m.shape == () and kept[1].shape == (3,) and torch.equal(y, ref[0][0]) and torch.equal(m, ref[1][0])
    g, g0 = gdr.gdr_norm_bwd(dy[0], kept, m, r), gdr.gdr_norm_bwd(dy, ref[3], ref[1], ref[2])
    assert torch.equal(g["x"], g0["x"][0]) and torch.equal(g["weight"], g0["weight"])
    with pytest.raises(gdr.GdrError):            # in place: refused
        gdr.gdr_norm_fwd(x, y=x)
    with pytest.raises(gdr.GdrError):            # no rows
        gdr.gdr_norm_fwd(x[:0])


def test_norm_other_stream_and_given_workspace():
    """A call on a side stream, with a workspace that held something else before."""
    import torch
    import recurrent_state_memory_amd as gdr
    d = inputs(600, 130, "f32", 50)
    x, dy, w = dev(d["x"]), dev(d["dy"]), dev(d["w"])
    _, m, r, _ = gdr.gdr_norm_fwd(x, w)
    ref = gdr.gdr_norm_bwd(dy, x, m, r, w)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, m2, r2, _ = gdr.gdr_norm_fwd(x, w, stream=side)
    got = gdr.gdr_norm_bwd(dy, x, m2, r2, w, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(ref[k], got[k]) for k in ref)
    with pytest.raises(ValueError, match="workspace"):
        gdr.gdr_norm_bwd(dy, x, m, r, w, workspace=ws[:100])


def test_norm_graph_and_repeat():
    import torch
    import recurrent_state_memory_amd as gdr
    ds = [inputs(500, 384, "bf16", 40 + i) for i in range(2)]
    x, dy, w = dev(ds[0]["x"], "bf16"), dev(ds[0]["dy"], "bf16"), dev(ds[0]["w"])

    def both():
        y, m, r, kept = gdr.gdr_norm_fwd(x, w, return_ckpt8=True)
        return y, gdr.gdr_norm_bwd(dy, kept, m, r, w)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gg = both()
    for i in (1, 0, 1):
        x.copy_(dev(ds[i]["x"], "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        ey, eg = both()
        torch.cuda.synchronize()
        assert torch.equal(gy, ey) and all(torch.equal(gg[k], eg[k]) for k in eg)
