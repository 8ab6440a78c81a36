"""Channelwise operators on tensors of more than 2^31 elements: what lies behind the
32-bit border has to equal what the same values give before it, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room():
    import torch
    yield
    torch.cuda.empty_cache()


def _randn(*shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def test_scan_many_rows():
    """33 batch rows of 8192 x 8192: the last one lies behind 2^31 elements."""
    import torch
    import recurrent_state_memory_amd as gdr
    bf = torch.bfloat16
    one = [_randn(1, 8192, 8192, dtype=bf, seed=i) for i in range(3)]
    A = torch.linspace(0.01, 1, 8192, device="cuda")
    x, d, dy = (t.expand(33, -1, -1).contiguous() for t in one)
    assert x.numel() > 1 << 31
    y, h, ck = gdr.gdr_scan_fwd_gated(x, d, A, return_ckpt=True)
    y1, h1, ck1 = gdr.gdr_scan_fwd_gated(one[0], one[1], A, return_ckpt=True)
    for b in (0, 31, 32):
        assert torch.equal(y[b], y1[0]) and torch.equal(h[b], h1[0]) and torch.equal(ck[b], ck1[0])
    del y
    g = gdr.gdr_scan_bwd_gated(x, d, A, dy, ckpt=ck)
    g1 = gdr.gdr_scan_bwd_gated(one[0], one[1], A, one[2], ckpt=ck1)
    for k in ("x", "decay_x", "h0"):
        assert torch.equal(g[k][32], g1[k][0]) and torch.equal(g[k][0], g1[k][0]), k


def test_scan_one_long_row():
    """One sequence of 270336 tokens x 8192 channels: its end, run again from the state in between."""
    import torch
    import recurrent_state_memory_amd as gdr
    T, cut, C = 270336, 1 << 18, 8192
    x = _randn(1, T, C, dtype=torch.bfloat16, seed=4)
    alpha = torch.rand((1, T, C), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    alpha.mul_(0.001).add_(0.999)
    y, h, _ = gdr.gdr_scan_fwd(x, alpha)
    ya, ha, _ = gdr.gdr_scan_fwd(x[:, :cut], alpha[:, :cut])
    assert torch.equal(ya[:, -64:], y[:, cut - 64:cut])
    yb, hb, _ = gdr.gdr_scan_fwd(x[:, cut:], alpha[:, cut:], h0=ha)
    assert torch.equal(yb, y[:, cut:]) and torch.equal(hb, h)


def test_norm_and_ckpt8_many_rows():
    """300000 rows of 8192, every one the first 1000 again."""
    import torch
    import recurrent_state_memory_amd as gdr
    R, D = 300000, 8192
    x0, dy0 = _randn(1000, D, dtype=torch.bfloat16, seed=6), _randn(1000, D, dtype=torch.bfloat16, seed=7)
    x = x0.repeat(R // 1000, 1)
    assert x.numel() > 1 << 31
    y, m, r, kept = gdr.gdr_norm_fwd(x, return_ckpt8=True)
    y0, m0, r0, kept0 = gdr.gdr_norm_fwd(x0, return_ckpt8=True)
    u8 = torch.uint8
    for s in (slice(0, 1000), slice(R - 1000, R)):
        assert torch.equal(y[s], y0) and torch.equal(m[s], m0) and torch.equal(r[s], r0)
        assert torch.equal(kept[0][s].view(u8), kept0[0].view(u8)) and torch.equal(kept[1][s], kept0[1])
    del y
    code, exp = gdr.gdr_ckpt8_pack(x)
    assert torch.equal(code[R - 1000:].view(u8), kept0[0].view(u8)) and torch.equal(exp[R - 1000:], kept0[1])
    back = gdr.gdr_ckpt8_unpack(code, exp)
    assert torch.equal(back[R - 1000:], gdr.gdr_ckpt8_unpack(*kept0))
    del back, code, exp
    g = gdr.gdr_norm_bwd(dy0.repeat(R // 1000, 1), kept, m, r, need_grad_weight=False, need_grad_bias=False)
    g0 = gdr.gdr_norm_bwd(dy0, kept0, m0, r0, need_grad_weight=False, need_grad_bias=False)
    assert torch.equal(g["x"][R - 1000:], g0["x"]) and torch.equal(g["x"][:1000], g0["x"])
