"""The channelwise recurrence's gates at the ends of their range: gradients compared
with the fp64 oracle within bounds that are relative to each value (tests/_chan.py)."""
import numpy as np
import pytest

from _chan import E, check, dev, gate_bounds, half_step, scan_error, scan_inputs
from oracle import scan
from synth.gen import bf16_round
from test_gpu_scan import call_bwd, check_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("kind", ["norm", "gate+norm"])
def test_scan_bwd_of_nearly_closed_inputs(kind, ck):
    """decay_x so low that 1 - a^2 comes near fp32's least normal number (2^-126 = 1.2e-38;
    here from 2.7e-38 on): sqrt(1 - a^2) is about 1e-19 to 1e-17 in the gradients, as it
    is in the forward."""
    B, T, C = 2, 70, 68
    d = scan_inputs((B, T), C, "f32", kind, seed=84)
    rng = np.random.default_rng(85)
    d["kw"]["d"] = rng.uniform(-86.5, -80, (B, T, C)).astype(np.float32)
    d["kw"]["A"] = rng.uniform(0.5, 1, C).astype(np.float32)
    check_bwd(d, "f32", d["h"], d["dh"], f"nearly closed {kind}/ckpt={ck}", ck=ck)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["gate", "gate+norm"])
@pytest.mark.parametrize("low,high", [(8, 30), (-30, -8), (-8, 8)])
def test_scan_bwd_of_saturated_gates(low, high, kind, io):
    """grad_gate_x = G b x (1 - sigmoid(gate_x)), relative to itself also where the gate
    is open and 1 - sigmoid(gate_x) is 1e-4 to 1e-13.

    The bound: G's own error, and b x (rb + 1), 1 - s (as a sigmoid of -gate_x, which is
    within what rb counts for the sigmoid) and two products, all relative."""
    import torch
    B, T, C = 2, 70, 68
    d = scan_inputs((B, T), C, io, kind, seed=abs(high))
    cast = bf16_round if io == "bf16" else (lambda z: z.astype(np.float32))
    d["kw"]["g"] = cast(np.random.default_rng(low + 99).uniform(low, high, (B, T, C)).astype(np.float32))
    g = call_bwd(d, io, h0=dev(d["h"]), grad_h=dev(d["dh"]))
    torch.cuda.synchronize()
    r = scan.backward(d["x"], d["dy"], d["dh"], h0=d["h"], **d["kw"])
    q, G = r["q"], r["G"]
    ra, rb = gate_bounds(q, d["kw"]["g"])
    af = np.concatenate([np.ones((B, 1, C)), q["a"][:, :0:-1]], 1)
    raf = np.concatenate([np.zeros((B, 1, C)), ra[:, :0:-1]], 1)
    NG = scan_error(af, d["dy"][:, ::-1].astype(np.float64), raf, 0.0, d["dh"].astype(np.float64))[0][:, ::-1]
    shut = 1.0 / (1.0 + np.exp(d["kw"]["g"].astype(np.float64)))
    want = G * q["b"] * d["x"] * shut
    gs = np.abs(q["b"] * d["x"]) * shut
    check(f"saturated {kind}/{io}/{low}..{high} dg", g["gate_x"], want,
          NG * gs + np.abs(G) * gs * (2 * rb + 4) * E + half_step(io) * np.abs(want))


@pytest.mark.parametrize("kind", ["gate", "gate+norm"])
def test_scan_bwd_of_infinite_gates(kind):
    """A gate at -Inf takes nothing in: its token's gradients of x and gate_x are 0, and x
    there reaches no other gradient.  At +Inf grad_gate_x is 0 but for fp32's least normal number
    (times G b x), and grad_x that of a gate at 80."""
    import torch
    d = scan_inputs((2, 70), 68, "f32", kind, seed=13)
    g = d["kw"]["g"]
    g[0, 3::5] = -np.inf
    g[1, 4::5] = np.inf
    out = call_bwd(d, "f32", h0=dev(d["h"]), grad_h=dev(d["dh"]))
    assert all(torch.isfinite(t).all() for t in out.values())
    assert (out["x"][0, 3::5] == 0).all() and (out["gate_x"][0, 3::5] == 0).all()
    assert (out["gate_x"][1, 4::5].abs() <= 1e-34).all()
    d["x"][0, 3::5] *= 2
    g[1, 4::5] = 80
    again = call_bwd(d, "f32", h0=dev(d["h"]), grad_h=dev(d["dh"]))
    g[1, 4::5] = np.inf
    for k in out:
        a, b = out[k], again[k]
        if k == "gate_x":
            a, b = (torch.where(torch.isinf(dev(g)), 0, t) for t in (a, b))
        assert torch.equal(a, b), k
