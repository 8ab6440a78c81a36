"""A NaN, or an Inf, in one place: the backward passes of the convolution, the selective scan
and the group norm take it along its channel (its group of its row) and into the sums that
it enters; everything else keeps its bits."""
import pytest

from tests import _mixer as m

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf")]


def _same(a, b, hit):
    import torch
    assert torch.equal(a[~hit], b[~hit])


# Rows cut into segments or not, one state a wave, two, and turns of 16; channel 65 is the last one
# of its workgroup, whose data lanes without a channel read too.
@pytest.mark.parametrize("T", [70, 700])
@pytest.mark.parametrize("N", [5, 16, 40])
@pytest.mark.parametrize("bad", BAD)
def test_selective_scan(T, N, bad):
    import torch
    import recurrent_state_memory_amd as gdr
    B, C, G = 2, 66, 1
    for gate in (False, True):
        d = m.ssm_inputs(B, T, C, N, G, "f32", 7 + T + N)
        t = {k: m.dev(d[k]) for k in d}

        def call(**new):
            u = dict(t, **new)
            args = (u["x"], u["dt"], u["A"], u["Bv"], u["Cv"])
            kw = dict(D=u["D"], z=u["z"] if gate else None, dt_bias=u["dt_bias"])
            ck = gdr.gdr_ssm_fwd(*args, h0=u["h0"], return_ckpt=True, **kw)[2]
            return gdr.gdr_ssm_bwd(u["dy"], *args, ckpt=ck, grad_h=u["dh"], **kw)
        ref = call()
        at, c = 40, 65
        for name in ("x", "dt", "dy", "z", "dh"):
            if name == "z" and not gate:
                continue
            v = t[name].clone()
            if name == "dh":
                v[1, c, 2] = bad
            else:
                v[1, at, c] = bad
            g = call(**{name: v})
            for k in ("x", "dt", "z"):
                if k in ref:                   # the channel of this row alone
                    hit = torch.zeros_like(ref[k], dtype=torch.bool)
                    hit[1, :, c] = True
                    _same(g[k], ref[k], hit)
            for k in ("A", "D", "dt_bias"):    # the channel's own sums
                hit = torch.zeros_like(ref[k], dtype=torch.bool)
                hit[c] = True
                _same(g[k], ref[k], hit)
            hit = torch.zeros_like(ref["h0"], dtype=torch.bool)
            hit[1, c] = True
            _same(g["h0"], ref["h0"], hit)
            # the vectors' sums: the adjoint's from the token back, the state's from it on
            hitB, hitC = (torch.zeros_like(ref["B"], dtype=torch.bool) for _ in range(2))
            if name == "x":
                hitB[1, at] = hitC[1, at:] = True
            elif name == "dt":
                hitB[1, :at + 1] = hitC[1, at:] = True
            elif name == "dh":
                hitB[1, :, :, 2] = True        # and the adjoint of the other states as it was
            else:
                hitB[1, :at + 1] = hitC[1, at] = True
            _same(g["B"], ref["B"], hitB)
            _same(g["C"], ref["C"], hitC)
            if name == "dy":                   # and where it goes it shows
                assert not bool(torch.isfinite(g["C"][1, at]).any()) and not bool(torch.isfinite(g["h0"][1, c]).any())
            if name == "x":
                assert not bool(torch.isfinite(g["B"][1, at]).any()) and not bool(torch.isfinite(g["D"][c]))


@pytest.mark.parametrize("K,silu", [(4, True), (4, False), (7, True)])
@pytest.mark.parametrize("bad", BAD)
def test_convolution(K, silu, bad):
    import torch
    import recurrent_state_memory_amd as gdr
    B, T, C = 2, 90, 37
    d = m.conv_inputs(B, T, C, K, "f32", K)
    t = {k: m.dev(d[k]) for k in d}

    def call(**new):
        u = dict(t, **new)
        return gdr.gdr_conv_bwd(u["dy"], u["x"], u["w"], u["b"], state=u["st"], grad_state=u["dst"], silu=silu)
    ref = call()
    at, c = 50, 36
    for name in ("x", "dy"):
        v = t[name].clone()
        v[1, at, c] = bad
        g = call(**{name: v})
        hit = torch.zeros_like(ref["x"], dtype=torch.bool)
        # x reaches the pre-activations of K tokens, each of which reaches the gradients of K
        lo, hi = (at - K + 1, at + 1) if name == "dy" else (at - K + 1, at + K) if silu else (0, 0)
        hit[1, lo:hi, c] = True
        _same(g["x"], ref["x"], hit)
        assert torch.equal(g["state"], ref["state"])
        own = torch.arange(C, device="cuda") == c
        assert torch.equal(g["weight"][~own], ref["weight"][~own]) and torch.equal(g["bias"][~own], ref["bias"][~own])
        assert not bool(torch.isfinite(g["weight"][c]).any())


@pytest.mark.parametrize("D", [3, 21, 100, 700, 5000])
@pytest.mark.parametrize("bad", BAD)
def test_group_norm(D, bad):
    import torch
    import recurrent_state_memory_amd as gdr
    R, G = 5, 3
    gen = torch.Generator(device="cuda").manual_seed(D)
    dy, x, z = (torch.randn(R, G * D, device="cuda", generator=gen) for _ in range(3))
    w, b = (torch.randn(G * D, device="cuda", generator=gen) for _ in range(2))

    def call(dy, x, z):
        _, mean, rstd = gdr.gdr_gnorm_fwd(x, G, w, b, z=z, silu=True)
        return gdr.gdr_gnorm_bwd(dy, x, mean, rstd, G, w, b, z=z, silu=True)
    ref = call(dy, x, z)
    hit = torch.zeros(R, G, D, dtype=torch.bool, device="cuda")
    hit[2, 1] = True
    hit, cols = hit.view(R, G * D), hit[2].reshape(-1)
    for i in range(3):
        v = [dy.clone(), x.clone(), z.clone()]
        v[i][2, D + D // 2] = bad
        g = call(*v)
        _same(g["x"], ref["x"], hit)
        _same(g["z"], ref["z"], hit)
        _same(g["weight"], ref["weight"], cols)
        _same(g["bias"], ref["bias"], cols)
        assert not bool(torch.isfinite(g["x"][hit]).any())
