"""The channelwise recurrence with its final state written over its start state
(h_out = h0): the tiles of a chain read the one while the last of them writes the other."""
import pytest

from _chan import dev, scan_inputs
from test_gpu_scan import call_fwd

pytestmark = pytest.mark.gpu


# two tiles of 256 tokens, all eight of a chain's first super, and more; one chain and many
@pytest.mark.parametrize("kind", ["alpha", "gate+norm"])
@pytest.mark.parametrize("B,T,C", [(1, 300, 64), (2, 2000, 2048), (3, 2048, 130), (2, 5000, 1000), (40, 700, 64)])
def test_scan_in_place(B, T, C, kind):
    import torch
    d = scan_inputs((B, T), C, "bf16", kind, seed=T + C)
    h0 = dev(d["h"])
    y, h, _ = call_fwd(d, "bf16", h0=h0)
    for _ in range(5):
        state = h0.clone()
        y2, h2, _ = call_fwd(d, "bf16", h0=state, h_out=state)
        assert h2 is state and torch.equal(h, h2) and torch.equal(y, y2)
