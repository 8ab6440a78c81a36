"""GPU parity of the short causal convolution against the fp64 oracle, element by element."""
import numpy as np
import pytest

from oracle import conv
from tests import _mixer as m

pytestmark = pytest.mark.gpu

SHAPES = [  # B, T, C, K, padded
    (1, 1, 1, 2, False), (2, 1, 8, 4, False), (1, 2, 3, 8, False), (3, 7, 16, 4, True), (2, 33, 40, 3, False),
    (1, 64, 512, 4, False), (2, 65, 513, 5, True), (1, 700, 1, 4, False), (5, 19, 130, 6, True), (1, 300, 24, 7, False),
    (2, 130, 2056, 2, True), (1, 4100, 12, 8, False), (40, 3, 9, 3, True), (1, 1025, 64, 4, False),
]


def _lens(B, T, padded):
    """Full, empty, one token, beyond the end, negative and in between."""
    return [(T, 0, 1, T // 2, T + 5, -3, T - 1)[b % 7] for b in range(B)] if padded else None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,K,padded", SHAPES)
def test_forward(B, T, C, K, padded, io):
    import recurrent_state_memory_amd as gdr
    act = (T + K) % 2 == 0
    d = m.conv_inputs(B, T, C, K, io, T * C)
    lens = _lens(B, T, padded)
    x = m.dev(d["x"], io)
    if padded:                       # nothing behind a row's end is read
        for b, n in enumerate(lens):
            x[b, max(n, 0):] = float("nan")
    y, st = gdr.gdr_conv_fwd(x, m.dev(d["w"]), m.dev(d["b"]), state=m.dev(d["st"], io), lens=m.as_int32(lens), silu=act)
    y_r, st_r, u = conv.forward(d["x"], d["w"], d["b"], d["st"], lens, act)
    m.check("y", y, y_r, m.conv_bounds(d, K, act, y_r, u, io)[1])
    m.check("state", st, st_r, 0.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,K,padded", SHAPES)
def test_backward(B, T, C, K, padded, io):
    import recurrent_state_memory_amd as gdr
    act = (T + K) % 2 == 0
    d = m.conv_inputs(B, T, C, K, io, T * C + 1)
    lens = _lens(B, T, padded)
    x, dy = m.dev(d["x"], io), m.dev(d["dy"], io)
    if padded:
        for b, n in enumerate(lens):
            x[b, max(n, 0):] = float("nan")
            dy[b, max(n, 0):] = float("inf")
    g = gdr.gdr_conv_bwd(dy, x, m.dev(d["w"]), m.dev(d["b"]), state=m.dev(d["st"], io), lens=m.as_int32(lens), silu=act,
                         grad_state=m.dev(d["dst"], io))
    r = conv.backward(d["dy"], d["x"], d["w"], d["b"], d["st"], lens, act, d["dst"])
    y_r, _, u = conv.forward(d["x"], d["w"], d["b"], d["st"], None, act)
    eu = m.conv_bounds(d, K, act, y_r, u, io)[0]
    ex, es, ew, eb = m.conv_bwd_bounds(d, r, K, act, eu, io, T + B + 300)
    m.check("dx", g["x"], r["dx"], ex)
    m.check("dstate", g["state"], r["dstate"], es)
    m.check("dw", g["weight"], r["dw"], ew)
    m.check("db", g["bias"], r["db"], eb)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,K", [(1, 1, 2), (1, 2048, 4), (7, 13, 3), (300, 24, 4), (3, 1000, 8)])
def test_step_continues_the_forward(N, C, K, io):
    """Tokens one by one, the state in place, give the forward's own results exactly."""
    import torch
    import recurrent_state_memory_amd as gdr
    T = 11
    d = m.conv_inputs(N, T, C, K, io, C)
    x, w, b, st = m.dev(d["x"], io), m.dev(d["w"]), m.dev(d["b"]), m.dev(d["st"], io)
    y, so = gdr.gdr_conv_fwd(x, w, b, state=st)
    ys = [gdr.gdr_conv_step(st, x[:, t].contiguous(), w, b) for t in range(T)]
    assert torch.equal(torch.stack(ys, 1), y) and torch.equal(st, so)
    y_r, _, u = conv.forward(d["x"], d["w"], d["b"], d["st"])
    m.check("y", torch.stack(ys, 1), y_r, m.conv_bounds(d, K, True, y_r, u, io)[1])


def test_optional_arguments():
    """No bias, no state, no state's gradient; outputs given; the state overwritten in place."""
    import torch
    import recurrent_state_memory_amd as gdr
    d = m.conv_inputs(2, 50, 33, 4, "bf16", 5)
    x, w, dy, st = m.dev(d["x"], "bf16"), m.dev(d["w"]), m.dev(d["dy"], "bf16"), m.dev(d["st"], "bf16")
    zb, zs = torch.zeros(33, device="cuda"), torch.zeros_like(st)
    y, so = gdr.gdr_conv_fwd(x, w)
    y0, so0 = gdr.gdr_conv_fwd(x, w, zb, state=zs)
    assert torch.equal(y, y0) and torch.equal(so, so0)
    assert gdr.gdr_conv_fwd(x, w, return_state=False)[1] is None
    g, g0 = gdr.gdr_conv_bwd(dy, x, w, need_grad_state=False), gdr.gdr_conv_bwd(dy, x, w, zb, state=zs, grad_state=zs)
    assert set(g) == {"x", "weight"} and set(g0) == {"x", "weight", "bias", "state"}
    assert torch.equal(g["x"], g0["x"]) and torch.equal(g["weight"], g0["weight"])
    out = torch.empty_like(x)
    y1, so1 = gdr.gdr_conv_fwd(x, w, state=st)
    r = gdr.gdr_conv_fwd(x, w, state=st, state_out=st, y=out)
    assert r[0] is out and r[1] is st and torch.equal(out, y1) and torch.equal(st, so1)


def test_pieces_of_a_sequence():
    """A call on each piece, the state handed on, gives one call's results."""
    import torch
    import recurrent_state_memory_amd as gdr
    d = m.conv_inputs(2, 90, 20, 4, "f32", 6)
    x, w, b = m.dev(d["x"]), m.dev(d["w"]), m.dev(d["b"])
    y, so = gdr.gdr_conv_fwd(x, w, b)
    st, ys = None, []
    for t0, t1 in ((0, 1), (1, 3), (3, 40), (40, 90)):
        yi, st = gdr.gdr_conv_fwd(x[:, t0:t1].contiguous(), w, b, state=st)
        ys.append(yi)
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(st, so)


def test_unaligned_buffers():
    """Any alignment of one element, and nothing outside the tensors is written."""
    import torch
    import recurrent_state_memory_amd as gdr
    B, T, C, K = 2, 21, 37, 4
    d = m.conv_inputs(B, T, C, K, "bf16", 7)
    w, b, n = m.dev(d["w"]), m.dev(d["b"]), B * T * C
    ref, _ = gdr.gdr_conv_fwd(m.dev(d["x"], "bf16"), w, b)
    gref = gdr.gdr_conv_bwd(m.dev(d["dy"], "bf16"), m.dev(d["x"], "bf16"), w, b)
    for off in (1, 3, 7):
        bx, by, bd = (torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        bx[off:off + n] = m.dev(d["x"], "bf16").flatten()
        bd[off:off + n] = m.dev(d["dy"], "bf16").flatten()
        x, y, dy = (t[off:off + n].view(B, T, C) for t in (bx, by, bd))
        gdr.gdr_conv_fwd(x, w, b, y=y)
        assert torch.equal(y, ref) and bool((by[:off] == 5).all()) and bool((by[off + n:] == 5).all())
        g = gdr.gdr_conv_bwd(dy, x, w, b)
        assert all(torch.equal(g[k], gref[k]) for k in g)
