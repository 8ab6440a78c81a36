"""The channelwise recurrence in the forms that test_gpu_scan.py leaves out: x in 8 bits
with every kind of gate, more chains than one team works on, steps of many states."""
import numpy as np
import pytest

from _chan import E, check, dev, gate_bounds, half_step, scan_inputs
from oracle import scan
from test_gpu_scan import call_fwd, check_bwd, check_fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("kind", ["decay", "gate", "norm"])
@pytest.mark.parametrize("shape", [(2, 45, 63), (1, 290, 132)], ids=str)
def test_scan_bwd_from_8_bits(shape, kind, ck, io):
    B, T, C = shape
    d = scan_inputs((B, T), C, io, kind, seed=T + C)
    check_bwd(d, io, d["h"], d["dh"], f"bwd8 {kind}/{io}/{shape}/ckpt={ck}", x8=True, ck=ck)


# teams of 32 chains (decays given, fp32) and of 128, the last one short; two to ten tiles
@pytest.mark.parametrize("shape,kind,io", [((35, 300, 64), "alpha", "bf16"), ((11, 1200, 200), "alpha", "f32"),
                                           ((37, 520, 66), "gate+norm", "f32"), ((131, 270, 64), "gate+norm", "bf16"),
                                           ((66, 1100, 130), "norm", "bf16")], ids=str)
def test_scan_last_team_of_chains(shape, kind, io):
    B, T, C = shape
    d = scan_inputs((B, T), C, io, kind, seed=B)
    check_fwd(d, io, d["h"], f"teams fwd {kind}/{io}/{shape}")
    for ck in (False, True):
        check_bwd(d, io, d["h"], d["dh"], f"teams bwd {kind}/{io}/{shape}/ckpt={ck}", ck=ck)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["alpha", "gate+norm"])
@pytest.mark.parametrize("N,C", [(1024, 1000), (300, 8192)])
def test_scan_step_of_many_states(N, C, kind, io):
    import torch
    import recurrent_state_memory_amd as gdr
    d = scan_inputs((N,), C, io, kind, seed=N)
    k = d["kw"]
    h = dev(d["h"])
    if "alpha" in k:
        y = gdr.gdr_scan_step(h, dev(d["x"], io), dev(k["alpha"]))
    else:
        y = gdr.gdr_scan_step_gated(h, dev(d["x"], io), dev(k["d"], io), dev(k["A"]), gate_x=dev(k["g"], io))
    torch.cuda.synchronize()
    want = scan.step(d["h"], d["x"], **k)
    q = scan.gates(**k)
    ra, rb = gate_bounds(q, k.get("g"))
    tol = q["a"] * np.abs(d["h"]) * (ra + 2) * E + np.abs(q["b"] * d["x"]) * (rb + 2) * E + E * np.abs(want)
    check(f"step {N}x{C} {kind}/{io} h", h, want, tol)
    check(f"step {N}x{C} {kind}/{io} y", y, want, tol + half_step(io) * np.abs(want))


@pytest.mark.parametrize("kind", ["alpha", "gate+norm"])
def test_scan_inf_stays_in_its_channel(kind):
    """An Inf in x or in the start state: its channel is not finite from there on, and
    every other value is the one without it, bit for bit."""
    import torch
    d = scan_inputs((2, 700), 70, "f32", kind, seed=10)
    clean = call_fwd(d, "f32", h0=dev(d["h"]))
    d["x"][1, 50, 33] = np.inf
    d["h"][0, 5] = -np.inf
    y, h, _ = call_fwd(d, "f32", h0=dev(d["h"]))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 50:, 33] = bad[0, :, 5] = True
    assert not torch.isfinite(y[bad]).any() and torch.equal(y[~bad], clean[0][~bad])
    assert torch.equal(torch.isfinite(h), ~bad[:, -1]) and torch.equal(h[~bad[:, -1]], clean[1][~bad[:, -1]])
