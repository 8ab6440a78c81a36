"""Workspaces of exactly the size that the queries name, in the middle of a larger buffer: the
results of an allocated one, nothing touched outside, a byte less refused."""
import pytest

from tests import _mixer as m

pytestmark = pytest.mark.gpu


@pytest.fixture
def needs(monkeypatch):
    """The sizes that calls ask for, in their order."""
    import recurrent_state_memory_amd as gdr
    asked, plain = [], gdr._workspace

    def spy(need, workspace, dev):
        asked.append(need)
        return plain(need, workspace, dev)
    monkeypatch.setattr(gdr, "_workspace", spy)
    return asked


def _check(call, needs):
    import torch
    ref = call()
    ref = ref if isinstance(ref, dict) else dict(enumerate(ref))
    need = needs[-1]
    if need == 0:
        return 0
    pad = 4096
    for fill in (0, 255):           # 255: NaN wherever a number is read that was not written
        buf = torch.full((need + 2 * pad,), fill, dtype=torch.uint8, device="cuda")
        got = call(workspace=buf[pad:pad + need])
        got = got if isinstance(got, dict) else dict(enumerate(got))
        for k in ref:
            assert ref[k] is None or torch.equal(got[k], ref[k]), (k, fill)
        assert bool((buf[:pad] == fill).all()) and bool((buf[pad + need:] == fill).all()), fill
    with pytest.raises(ValueError, match="workspace"):
        call(workspace=buf[pad:pad + need - 1])
    return need


# Sizes whose forward and backward cut rows into different numbers of segments (200: 1 and
# several, 1500: 23 and others), every number of states a wave, groups, lanes without a channel.
@pytest.mark.parametrize("B,T,C,N,G", [(1, 1500, 20, 33, 2), (1, 200, 64, 16, 1), (2, 300, 70, 1, 1), (3, 90, 66, 5, 2),
                                       (2, 700, 130, 9, 1), (4, 130, 40, 17, 4), (1, 64, 3, 64, 3), (130, 40, 5, 3, 1)])
def test_selective_scan(B, T, C, N, G, needs):
    import torch
    import recurrent_state_memory_amd as gdr
    d = m.ssm_inputs(B, T, C, N, G, "f32", T + N)
    t = {k: m.dev(d[k]) for k in d}
    args = (t["x"], t["dt"], t["A"], t["Bv"], t["Cv"])
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], lens=m.as_int32([T - b % 3 * (T // 3) for b in range(B)]))
    _check(lambda **k: gdr.gdr_ssm_fwd(*args, h0=t["h0"], return_ckpt=True, **kw, **k), needs)
    ck = gdr.gdr_ssm_fwd(*args, h0=t["h0"], return_ckpt=True, **kw)[2]
    sizes = [_check(lambda **k: gdr.gdr_ssm_bwd(t["dy"], *args, grad_h=t["dh"], **start, **kw, **k), needs)
             for start in (dict(h0=t["h0"]), dict(ckpt=ck))]
    assert sizes[0] > sizes[1] > 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("B,T,C,K", [(2, 600, 72, 4), (1, 9, 3, 8), (3, 1001, 333, 3), (1, 4100, 12, 2), (40, 70, 520, 5)])
def test_convolution(B, T, C, K, needs):
    import recurrent_state_memory_amd as gdr
    d = m.conv_inputs(B, T, C, K, "bf16", T)
    t = {k: m.dev(d[k], None if k in "wb" else "bf16") for k in d}
    assert _check(lambda **k: gdr.gdr_conv_bwd(t["dy"], t["x"], t["w"], t["b"], state=t["st"], grad_state=t["dst"], **k), needs)


@pytest.mark.parametrize("R,G,D", [(1, 1, 1), (700, 2, 3), (513, 1, 64), (5, 3, 100), (33, 2, 5000), (2000, 16, 8), (3, 1, 16384)])
def test_group_norm(R, G, D, needs):
    import torch
    import recurrent_state_memory_amd as gdr
    gen = torch.Generator(device="cuda").manual_seed(R)
    dy, x, z = (torch.randn(R, G * D, device="cuda", generator=gen) for _ in range(3))
    w, b = (torch.randn(G * D, device="cuda", generator=gen) for _ in range(2))
    _, mean, rstd = gdr.gdr_gnorm_fwd(x, G, w, b, z=z, silu=True)
    assert _check(lambda **k: gdr.gdr_gnorm_bwd(dy, x, mean, rstd, G, w, b, z=z, silu=True, **k), needs)
