"""The convolution, the selective scan and the gated group norm on tensors of more than 2^31
elements or bytes a row: what lies behind the 32-bit borders has to equal what the same
values give before them."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room():
    import torch
    yield
    torch.cuda.empty_cache()


def _randn(*shape, seed, dtype=None):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype or torch.bfloat16)


def test_conv_many_rows():
    """33 batch rows of 8192 x 8192: the last one lies behind 2^31 elements."""
    import torch
    import recurrent_state_memory_amd as gdr
    x1, dy1 = _randn(1, 8192, 8192, seed=1), _randn(1, 8192, 8192, seed=2)
    w, b = _randn(8192, 4, seed=3, dtype=torch.float32), _randn(8192, seed=4, dtype=torch.float32)
    x = x1.expand(33, -1, -1).contiguous()
    assert x.numel() > 1 << 31
    y, st = gdr.gdr_conv_fwd(x, w, b)
    y1, st1 = gdr.gdr_conv_fwd(x1, w, b)
    for r in (0, 31, 32):
        assert torch.equal(y[r], y1[0]) and torch.equal(st[r], st1[0])
    del y
    g = gdr.gdr_conv_bwd(dy1.expand(33, -1, -1).contiguous(), x, w, b)
    g1 = gdr.gdr_conv_bwd(dy1, x1, w, b)
    for r in (0, 31, 32):
        assert torch.equal(g["x"][r], g1["x"][0]) and torch.equal(g["state"][r], g1["state"][0])


def test_gnorm_many_rows():
    """300000 rows of 8192, every one the first 1000 again."""
    import torch
    import recurrent_state_memory_amd as gdr
    R, C, G = 300000, 8192, 64
    x0, z0, dy0 = (_randn(1000, C, seed=5 + i) for i in range(3))
    x, z = x0.repeat(R // 1000, 1), z0.repeat(R // 1000, 1)
    assert x.numel() > 1 << 31
    y, m, r = gdr.gdr_gnorm_fwd(x, G, z=z, silu=True)
    y0, m0, r0 = gdr.gdr_gnorm_fwd(x0, G, z=z0, silu=True)
    for s in (slice(0, 1000), slice(R - 1000, R)):
        assert torch.equal(y[s], y0) and torch.equal(m[s], m0) and torch.equal(r[s], r0)
    del y
    g = gdr.gdr_gnorm_bwd(dy0.repeat(R // 1000, 1), x, m, r, G, z=z, silu=True, need_grad_weight=False, need_grad_bias=False)
    g0 = gdr.gdr_gnorm_bwd(dy0, x0, m0, r0, G, z=z0, silu=True, need_grad_weight=False, need_grad_bias=False)
    for s in (slice(0, 1000), slice(R - 1000, R)):
        assert torch.equal(g["x"][s], g0["x"]) and torch.equal(g["z"][s], g0["z"])


def test_ssm_many_rows():
    """33 batch rows of 8192 x 8192: the last one lies behind 2^31 elements."""
    import torch
    import recurrent_state_memory_amd as gdr
    C, T, N = 8192, 8192, 8
    one = [_randn(1, T, C, seed=10 + i) for i in range(3)]
    vec = [_randn(1, T, 1, N, seed=20 + i) for i in range(2)]
    A = -torch.rand(C, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    bias = torch.full((C,), -4.0, device="cuda")
    x, dt, dy, Bv, Cv = (v.expand(33, *v.shape[1:]).contiguous() for v in one + vec)
    assert x.numel() > 1 << 31
    y, h, ck = gdr.gdr_ssm_fwd(x, dt, A, Bv, Cv, dt_bias=bias, return_ckpt=True)
    y2, h2, ck2 = gdr.gdr_ssm_fwd(*(v[:4] for v in (x, dt)), A, *(v[:4] for v in (Bv, Cv)), dt_bias=bias, return_ckpt=True)
    for r in (0, 31, 32):
        assert torch.equal(y[r], y2[0]) and torch.equal(h[r], h2[0]) and torch.equal(ck[r], ck2[0])
    del y, y2
    g = gdr.gdr_ssm_bwd(dy, x, dt, A, Bv, Cv, dt_bias=bias, ckpt=ck)
    for k in ("x", "dt", "B", "C", "h0"):
        assert torch.equal(g[k][32], g[k][0]) and torch.equal(g[k][31], g[k][0]), k
    assert bool(torch.isfinite(g["A"]).all())


def test_ssm_rows_beyond_a_descriptor():
    """One sequence whose rows are 3.2 GB: segments split it whatever the chains, and pieces
    of it give the same to the rounding of the segments' joins."""
    import torch
    import recurrent_state_memory_amd as gdr
    T, cut, C, N = 98304, 65536, 16384, 4
    x, dt = _randn(1, T, C, seed=30), _randn(1, T, C, seed=31)
    Bv, Cv = _randn(1, T, 1, N, seed=32), _randn(1, T, 1, N, seed=33)
    A = -torch.rand(C, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) - 0.1
    bias = torch.full((C,), -4.0, device="cuda")
    y, h, _ = gdr.gdr_ssm_fwd(x, dt, A, Bv, Cv, dt_bias=bias)
    ya, ha, _ = gdr.gdr_ssm_fwd(x[:, :cut], dt[:, :cut], A, Bv[:, :cut], Cv[:, :cut], dt_bias=bias)
    yb, hb, _ = gdr.gdr_ssm_fwd(x[:, cut:], dt[:, cut:], A, Bv[:, cut:], Cv[:, cut:], dt_bias=bias, h0=ha)
    # a state's relative error: as many roundings as it has tokens behind it that still count,
    # 2^-24 each; decays of 0.1 * softplus(-4 + noise) forget within some 2^13 tokens
    scale = float(h.abs().max())
    assert float((h - hb).abs().max()) <= 2.0 ** -11 * scale
    for got, part in ((y[:, :cut], ya), (y[:, cut:], yb)):
        top = float(part.abs().max())
        for t in range(0, part.shape[1], 8192):
            assert float((got[:, t:t + 8192].float() - part[:, t:t + 8192].float()).abs().max()) <= (2.0 ** -8 + 2.0 ** -11) * top
    del y, ya, yb
    dy = _randn(1, T, C, seed=34)
    g = gdr.gdr_ssm_bwd(dy, x, dt, A, Bv, Cv, dt_bias=bias)
    gb = gdr.gdr_ssm_bwd(dy[:, cut:], x[:, cut:], dt[:, cut:], A, Bv[:, cut:], Cv[:, cut:], dt_bias=bias, h0=ha)
    for k in ("x", "dt", "B", "C"):
        top = float(gb[k].abs().max())
        for t in range(0, T - cut, 8192):
            a, b = g[k][:, cut + t:cut + t + 8192].float(), gb[k][:, t:t + 8192].float()
            assert float((a - b).abs().max()) <= (2.0 ** -8 + 2.0 ** -11) * top, k
