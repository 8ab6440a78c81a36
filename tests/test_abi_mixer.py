"""The convolution's, the selective scan's and the gated group norm's entry points without a
GPU: struct layouts, refusals before any HIP call, the binding's own checks."""
import ctypes
import os
import subprocess

import pytest

import recurrent_state_memory_amd as gdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def P(i, off=0):
    """A fake pointer, far from the others, never dereferenced: refusals come first."""
    return ((i + 1) << 40) + off


STRUCTS = {"gdr_conv_args": gdr.ConvArgs, "gdr_conv_bwd_args": gdr.ConvBwdArgs, "gdr_conv_step_args": gdr.ConvStepArgs,
           "gdr_ssm_args": gdr.SsmArgs, "gdr_ssm_bwd_args": gdr.SsmBwdArgs, "gdr_ssm_step_args": gdr.SsmStepArgs,
           "gdr_gnorm_args": gdr.GnormArgs, "gdr_gnorm_bwd_args": gdr.GnormBwdArgs}


def test_struct_layouts_match_the_headers(tmp_path):
    lines = ["#include <cstddef>", "#include <cstdio>", '#include "gdr_conv.h"', '#include "gdr_ssm.h"',
             '#include "gdr_gnorm.h"', "int main() {"]
    for c, s in STRUCTS.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in s._fields_]
    lines.append('printf("BLOCK %d\\n", GDR_SSM_BLOCK); return 0; }')
    src, exe = tmp_path / "l.cpp", tmp_path / "l"
    src.write_text("\n".join(lines))
    subprocess.run(["g++", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, s in STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(s), c
        for f, _ in s._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(s, f).offset, (c, f)
    assert int(got["BLOCK"]) == gdr.GDR_SSM_BLOCK


N, OK = gdr.GDR_ERR_NULL, gdr.GDR_OK
S, A, U, D, L, W = (gdr.GDR_ERR_SHAPE, gdr.GDR_ERR_ARG, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_ERR_DTYPE, gdr.GDR_ERR_ALIGN,
                    gdr.GDR_ERR_WORKSPACE)


def refuse(name, cls, base, cases):
    for kw, status in cases:
        assert gdr.call_channelwise(name, cls(**{**base, **kw})) == status, (name, kw)


SIZES = [(dict(B=0), S), (dict(T=0), S), (dict(C=-1), S), (dict(io_dtype=2), D), (dict(C=(1 << 18) + 4), U),
         (dict(B=1 << 15, T=1 << 15), S), (dict(B=1, T=(1 << 30) - 1, C=1028), S)]


def test_conv_refusals():
    n = 2 * 100 * 66 * 2
    base = dict(B=2, T=100, C=66, K=4, io_dtype=gdr.GDR_BF16, silu=1, x=P(0), weight=P(1), y=P(2))
    refuse("gdr_conv_fwd", gdr.ConvArgs, base, SIZES + [
        (dict(x=None), N), (dict(weight=None), N), (dict(y=None), N), (dict(K=1), U), (dict(K=9), U), (dict(K=0), S),
        (dict(silu=2), A), (dict(B=1 << 22, T=1, C=1), U), (dict(x=P(0, 1)), L), (dict(weight=P(1, 2)), L),
        (dict(bias=P(3, 1)), L), (dict(lens=P(4, 2)), L), (dict(state=P(5, 1)), L), (dict(y=P(0)), A),
        (dict(y=P(0, n - 2)), A), (dict(state=P(5), state_out=P(5, 2)), A), (dict(state_out=P(2, 64)), A),
        (dict(state_out=P(4), lens=P(4, 4)), A)])
    base = dict(B=2, T=100, C=66, K=4, io_dtype=gdr.GDR_BF16, silu=1, x=P(0), weight=P(1), grad_y=P(2), grad_x=P(6),
                grad_weight=P(7), workspace=P(30), workspace_bytes=1 << 30)
    refuse("gdr_conv_bwd", gdr.ConvBwdArgs, base, SIZES + [
        (dict(x=None), N), (dict(weight=None), N), (dict(grad_y=None), N), (dict(grad_x=None), N), (dict(grad_weight=None), N),
        (dict(K=9), U), (dict(silu=-1), A), (dict(grad_x=P(2)), A), (dict(grad_bias=P(7, 16)), A),
        (dict(grad_state=P(8), grad_state_out=P(8)), A), (dict(workspace=P(30, 8)), L), (dict(workspace=None), W),
        (dict(workspace_bytes=16), W), (dict(grad_x=P(6, 1)), L)])
    base = dict(N=4, C=66, K=4, io_dtype=gdr.GDR_F32, silu=0, x=P(0), weight=P(1), state=P(2), state_out=P(2), y=P(3))
    refuse("gdr_conv_step", gdr.ConvStepArgs, base, [
        (dict(x=None), N), (dict(weight=None), N), (dict(state=None), N), (dict(state_out=None), N), (dict(y=None), N),
        (dict(N=0), S), (dict(N=1 << 21, C=1 << 9), S), (dict(K=1), U), (dict(io_dtype=7), D), (dict(reserved=1), A),
        (dict(state_out=P(2, 4)), A), (dict(y=P(2)), A), (dict(y=P(0)), A), (dict(state=P(2, 2)), L)])


def test_ssm_refusals():
    base = dict(B=2, T=100, C=66, N=16, G=3, io_dtype=gdr.GDR_BF16, softplus=1, x=P(0), dt=P(1), A=P(2), Bv=P(3), Cv=P(4),
                y=P(5), workspace=P(30), workspace_bytes=1 << 30)
    missing = [(dict([(k, None)]), N) for k in ("x", "dt", "A", "Bv", "Cv")]
    shapes = [(dict(N=0), S), (dict(G=0), S), (dict(G=4), S), (dict(N=65), U), (dict(softplus=2), A), (dict(reserved=1), A),
              (dict(B=1 << 21, T=1), U)]
    refuse("gdr_ssm_fwd", gdr.SsmArgs, base, SIZES[:4] + missing + shapes + [
        (dict(y=None), N), (dict(x=P(0, 1)), L), (dict(A=P(2, 2)), L), (dict(D=P(6, 1)), L), (dict(h0=P(7, 2)), L),
        (dict(lens=P(8, 1)), L), (dict(workspace=P(30, 4)), L), (dict(y=P(0)), A), (dict(y=P(3, 2)), A),
        (dict(h0=P(7), h_out=P(7, 4)), A), (dict(ckpt=P(5, 64)), A),
        (dict(T=4096, workspace=None), W), (dict(T=4096, workspace_bytes=256), W)])       # segments side by side
    base = dict(base, y=None, grad_y=P(5), grad_x=P(10), grad_dt=P(11), grad_A=P(12), grad_Bv=P(13), grad_Cv=P(14))
    del base["y"]
    refuse("gdr_ssm_bwd", gdr.SsmBwdArgs, base, SIZES[:4] + missing + shapes + [
        (dict([(k, None)]), N) for k in ("grad_y", "grad_x", "grad_dt", "grad_A", "grad_Bv", "grad_Cv")] + [
        (dict(D=P(6)), N), (dict(z=P(6)), N), (dict(dt_bias=P(6)), N), (dict(grad_D=P(6)), A), (dict(grad_z=P(6)), A),
        (dict(grad_dt_bias=P(6)), A), (dict(h0=P(7), ckpt=P(8)), A), (dict(grad_x=P(5)), A), (dict(grad_Bv=P(14, 2)), A),
        (dict(grad_h0=P(12)), A), (dict(workspace=None), W), (dict(workspace_bytes=4096), W), (dict(grad_A=P(12, 2)), L)])
    base = dict(R=4, C=66, N=16, G=1, io_dtype=gdr.GDR_F32, softplus=1, x=P(0), dt=P(1), A=P(2), Bv=P(3), Cv=P(4), h=P(5),
                h_out=P(5), y=P(6))
    refuse("gdr_ssm_step", gdr.SsmStepArgs, base, missing + [
        (dict(h=None), N), (dict(h_out=None), N), (dict(y=None), N), (dict(R=0), S), (dict(G=4), S), (dict(N=65), U),
        (dict(R=1 << 13, C=1 << 14), S), (dict(io_dtype=-1), D), (dict(softplus=3), A), (dict(h_out=P(5, 4)), A),
        (dict(y=P(5)), A), (dict(y=P(0)), A), (dict(h=P(5, 2)), L)])


def test_gnorm_refusals():
    base = dict(R=5, C=120, G=4, io_dtype=gdr.GDR_F32, center=1, silu=0, eps=1e-5, x=P(0), y=P(1))
    shapes = [(dict(R=0), S), (dict(C=0), S), (dict(G=0), S), (dict(G=7), S), (dict(R=1 << 30), S), (dict(G=1, C=16385), U),
              (dict(G=1 << 10, C=(1 << 20) + 1024), U), (dict(io_dtype=3), D), (dict(silu=2), A)]
    refuse("gdr_gnorm_fwd", gdr.GnormArgs, base, shapes + [
        (dict(x=None), N), (dict(y=None), N), (dict(center=2), A), (dict(eps=-1.0), A), (dict(eps=float("nan")), A),
        (dict(eps=float("inf")), A), (dict(center=0, mean=P(3)), A), (dict(y=P(0)), A), (dict(z=P(1, 8)), A),
        (dict(mean=P(3), rstd=P(3, 16)), A), (dict(x=P(0, 2)), L), (dict(weight=P(4, 1)), L)])
    base = dict(R=5, C=120, G=4, io_dtype=gdr.GDR_BF16, silu=0, x=P(0), rstd=P(1), grad_y=P(2), grad_x=P(3), grad_weight=P(4),
                grad_bias=P(5), workspace=P(30), workspace_bytes=1 << 30)
    refuse("gdr_gnorm_bwd", gdr.GnormBwdArgs, base, shapes + [
        (dict(x=None), N), (dict(rstd=None), N), (dict(grad_y=None), N), (dict(grad_x=None), N), (dict(z=P(6)), N),
        (dict(grad_z=P(6)), A), (dict(grad_x=P(0)), A), (dict(grad_bias=P(4)), A), (dict(grad_y=P(2, 1)), L),
        (dict(workspace=P(30, 4)), L), (dict(workspace=None), W), (dict(workspace_bytes=32), W)])


def test_null_structs_and_workspace_queries():
    lib = gdr.load_library()
    for name in ("gdr_conv_fwd", "gdr_conv_bwd", "gdr_conv_step", "gdr_ssm_fwd", "gdr_ssm_bwd", "gdr_ssm_step",
                 "gdr_gnorm_fwd", "gdr_gnorm_bwd"):
        assert getattr(lib, name)(None, None) == N
    for name in ("gdr_conv_bwd_workspace", "gdr_ssm_fwd_workspace", "gdr_ssm_bwd_workspace", "gdr_gnorm_bwd_workspace"):
        assert getattr(lib, name)(None) == 0
    q = dict(B=2, C=66, N=16, G=3, io_dtype=1, softplus=1, x=P(0), dt=P(1), A=P(2), Bv=P(3), Cv=P(4), y=P(5))
    need = lib.gdr_ssm_fwd_workspace
    assert need(ctypes.byref(gdr.SsmArgs(**q, T=255))) == 0 and need(ctypes.byref(gdr.SsmArgs(**q, T=256))) > 0
    assert need(ctypes.byref(gdr.SsmArgs(**dict(q, B=200), T=4096))) == 0 and need(ctypes.byref(gdr.SsmArgs(**q, T=0))) == 0
    q = dict(R=5, C=120, G=4, io_dtype=1, silu=0, x=P(0), rstd=P(1), grad_y=P(2), grad_x=P(3))
    need = lib.gdr_gnorm_bwd_workspace
    assert need(ctypes.byref(gdr.GnormBwdArgs(**q))) == 0                       # no columns' sums
    assert need(ctypes.byref(gdr.GnormBwdArgs(**q, grad_bias=P(4)))) > 0
    assert need(ctypes.byref(gdr.GnormBwdArgs(**dict(q, x=None), grad_bias=P(4)))) == 0


def test_binding_checks():
    """Shapes, types and contiguity are refused by name before the device is looked at;
    good arguments on the CPU get as far as the device."""
    import torch
    bf = torch.bfloat16
    x, w, v, A = torch.zeros(2, 5, 8, dtype=bf), torch.zeros(8, 4), torch.zeros(2, 5, 2, 3, dtype=bf), torch.zeros(8, 3)
    st, c, h, lens = torch.zeros(2, 3, 8, dtype=bf), torch.zeros(8), torch.zeros(2, 8, 3), torch.zeros(2, dtype=torch.int32)
    x1, v1, r = x[:, 0].contiguous(), v[:, 0].contiguous(), torch.zeros(2, 5, 2)
    calls = [
        ("GPU", lambda: gdr.gdr_conv_fwd(x, w, c, state=st, lens=lens)),
        ("GPU", lambda: gdr.gdr_conv_bwd(x, x, w, c, state=st, lens=lens, grad_state=st)),
        ("GPU", lambda: gdr.gdr_conv_step(st, x1, w, c)),
        ("GPU", lambda: gdr.gdr_ssm_fwd(x, x, A, v, v, D=c, z=x, dt_bias=c, h0=h, lens=lens)),
        ("GPU", lambda: gdr.gdr_ssm_bwd(x, x, x, A, v, v, D=c, z=x, dt_bias=c, h0=h, lens=lens, grad_h=h)),
        ("GPU", lambda: gdr.gdr_ssm_step(h, x1, x1, A, v1, v1, D=c, z=x1, dt_bias=c)),
        ("GPU", lambda: gdr.gdr_gnorm_fwd(x, 2, c, c, z=x)),
        ("GPU", lambda: gdr.gdr_gnorm_bwd(x, x, r, r, 2, c, c, z=x)),
        ("B,T,C", lambda: gdr.gdr_conv_fwd(x1, w)),
        ("C,K", lambda: gdr.gdr_conv_fwd(x, c)),
        ("weight", lambda: gdr.gdr_conv_fwd(x, w.to(bf))),
        ("weight", lambda: gdr.gdr_conv_fwd(x, torch.zeros(4, 8).t())),
        ("state", lambda: gdr.gdr_conv_fwd(x, w, state=st.float())),
        ("state", lambda: gdr.gdr_conv_step(st[:, :2].contiguous(), x1, w)),
        ("lens", lambda: gdr.gdr_conv_fwd(x, w, lens=lens.long())),
        ("contiguous", lambda: gdr.gdr_conv_fwd(x.transpose(0, 1), w)),
        ("grad_state", lambda: gdr.gdr_conv_bwd(x, x, w, grad_state=st[:1])),
        ("x has shape", lambda: gdr.gdr_conv_bwd(x, x[:1], w)),
        ("N,C", lambda: gdr.gdr_conv_step(st, x, w)),
        ("bfloat16 or float32", lambda: gdr.gdr_conv_fwd(x.half(), w)),
        ("A must", lambda: gdr.gdr_ssm_fwd(x, x, c, v, v)),
        ("A has", lambda: gdr.gdr_ssm_fwd(x, x, A[:4], v, v)),
        ("dt has", lambda: gdr.gdr_ssm_fwd(x, x.float(), A, v, v)),
        (r"B must be \[B,T,G,N\]", lambda: gdr.gdr_ssm_fwd(x, x, A, v1, v)),
        (r"B must be \[R,G,N\]", lambda: gdr.gdr_ssm_step(h, x1, x1, A, v, v)),
        ("C has shape", lambda: gdr.gdr_ssm_fwd(x, x, A, v, v[:, :, :1])),
        ("B has shape", lambda: gdr.gdr_ssm_fwd(x, x, A, v[..., :2].contiguous(), v)),
        ("z has", lambda: gdr.gdr_ssm_fwd(x, x, A, v, v, z=x[:1])),
        ("h0", lambda: gdr.gdr_ssm_fwd(x, x, A, v, v, h0=h.to(bf))),
        ("not both", lambda: gdr.gdr_ssm_bwd(x, x, x, A, v, v, h0=h, ckpt=torch.zeros(2, 1, 3, 8))),
        ("ckpt", lambda: gdr.gdr_ssm_bwd(x, x, x, A, v, v, ckpt=torch.zeros(2, 1, 8, 3))),
        ("h has", lambda: gdr.gdr_ssm_step(h[:1], x1, x1, A, v1, v1)),
        ("fall into", lambda: gdr.gdr_gnorm_fwd(x, 3)),
        ("fall into", lambda: gdr.gdr_gnorm_bwd(x, x, r, r, 0)),
        ("weight", lambda: gdr.gdr_gnorm_fwd(x, 2, c[:4])),
        ("z has", lambda: gdr.gdr_gnorm_fwd(x, 2, z=x.float())),
        ("rstd", lambda: gdr.gdr_gnorm_bwd(x, x, r, None, 2)),
        ("mean", lambda: gdr.gdr_gnorm_bwd(x, x, r[:, :1], r, 2)),
    ]
    for match, call in calls:
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("groups", [2.5, 2.0, "2", None])
def test_groups_are_whole(groups):
    import torch
    x, r = torch.zeros(3, 8), torch.zeros(3, 2)
    with pytest.raises(TypeError):
        gdr.gdr_gnorm_fwd(x, groups)
    with pytest.raises(TypeError):
        gdr.gdr_gnorm_bwd(x, x, r, r, groups)


def test_host_half_under_sanitizers(tmp_path):
    import shutil
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "harness"
    csrc = os.path.join(ROOT, "recurrent_state_memory_amd", "csrc")
    cmd = [gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
           "-I" + csrc, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g",
           os.path.join(ROOT, "tests", "mixer_host_harness.cpp"), os.path.join(csrc, "conv_api.cpp"),
           os.path.join(csrc, "ssm_api.cpp"), os.path.join(csrc, "gnorm_api.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "sanitizer" in r.stderr.lower():
        pytest.skip("sanitizer runtime not available: " + r.stderr[-200:])
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1:verify_asan_link_order=0")
    out = subprocess.run([str(exe)], capture_output=True, text=True, env=env)
    assert out.returncode == 0 and "MIXER_HARNESS_OK" in out.stdout, out.stdout + out.stderr
