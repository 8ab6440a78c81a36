"""The channelwise recurrence's gates at the ends of their range: gradients compared
with the fp64 oracle within bounds that are relative to each value (tests/_chan.py)."""
import numpy as np
import pytest

from _chan import scan_inputs
from test_gpu_scan import check_bwd

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
