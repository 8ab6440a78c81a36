"""Layer norm at row lengths and counts where the kernels' shapes change, between those
of test_gpu_norm.py: rows of two waves in odd numbers, with and without the 8-bit copy."""
import numpy as np
import pytest

from _chan import check, dev, norm_bounds
from oracle import norm
from test_gpu_norm import inputs
from test_gpu_norm import test_norm_bwd as check_norm_bwd
from test_gpu_norm import test_norm_fwd as check_norm_fwd

pytestmark = pytest.mark.gpu

# 128 threads a row: bf16 from 2049 values on (with the 8-bit copy from 1025), fp32 from
# 1025 on (513)
SHAPES = [(1, 700), (3, 700), (3, 1281), (3, 1300), (1, 2100), (257, 2500), (511, 1100)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", SHAPES)
def test_norm_fwd_rows_of_two_waves(R, D, io):
    import torch
    import recurrent_state_memory_amd as gdr
    check_norm_fwd(R, D, io)        # weights with the 8-bit copy, and neither
    d = inputs(R, D, io, R + D)
    plain = gdr.gdr_norm_fwd(dev(d["x"], io), dev(d["w"]), dev(d["b"]))
    torch.cuda.synchronize()
    yr, mr, rr = norm.forward(d["x"], d["w"], d["b"])
    ty, tm, tr = norm_bounds(d["x"].astype(np.float64), d["w"], mr, rr, 1e-5, yr, io)
    for name, got, want, tol in zip(("y", "mean", "rstd"), plain, (yr, mr, rr), (ty, tm, tr)):
        check(f"norm fwd {R}x{D}/{io} without the copy: {name}", got, want, tol)
    assert plain[3] is None


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,D", SHAPES)
def test_norm_bwd_rows_of_two_waves(R, D, io, x8):
    check_norm_bwd(R, D, io, x8)


@pytest.mark.parametrize("R,D", [(3, 10000), (300, 9001)])
def test_norm_bwd_three_runs_of_1024_threads(R, D):
    for x8 in (False, True):
        check_norm_bwd(R, D, "f32", x8)
