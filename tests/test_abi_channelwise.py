"""The channelwise entry points without a GPU: struct layouts, refusals before any
HIP call, the binding's own checks."""
import ctypes
import os
import subprocess

import pytest

import recurrent_state_memory_amd as gdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def P(i, off=0):
    """A fake pointer, far from the others, never dereferenced: refusals come first."""
    return ((i + 1) << 40) + off


STRUCTS = {"gdr_scan_args": gdr.ScanArgs, "gdr_scan_bwd_args": gdr.ScanBwdArgs,
           "gdr_scan_step_args": gdr.ScanStepArgs, "gdr_norm_args": gdr.NormArgs,
           "gdr_norm_bwd_args": gdr.NormBwdArgs, "gdr_ckpt8_pack_args": gdr.Ckpt8PackArgs,
           "gdr_ckpt8_unpack_args": gdr.Ckpt8UnpackArgs}


def test_struct_layouts_match_the_headers(tmp_path):
    lines = ["#include <cstddef>", "#include <cstdio>", '#include "gdr_scan.h"', '#include "gdr_norm.h"',
             '#include "gdr_ckpt8.h"', "int main() {"]
    for c, s in STRUCTS.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in s._fields_]
    lines.append(f'printf("BLOCK %d\\nGROUP %d\\n", GDR_SCAN_BLOCK, GDR_CKPT8_GROUP); return 0; }}')
    src, exe = tmp_path / "l.cpp", tmp_path / "l"
    src.write_text("\n".join(lines))
    subprocess.run(["g++", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, s in STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(s), c
        for f, _ in s._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(s, f).offset, (c, f)
    assert int(got["BLOCK"]) == gdr.GDR_SCAN_BLOCK and int(got["GROUP"]) == gdr.GDR_CKPT8_GROUP


def _fwd(**kw):
    d = dict(B=2, T=100, C=66, io_dtype=gdr.GDR_BF16, x=P(0), alpha=P(1), y=P(2), workspace=P(30),
             workspace_bytes=1 << 30)
    return gdr.ScanArgs(**{**d, **kw})


GATED = dict(alpha=None, decay_x=P(3), decay_a=P(4))
N, OK = gdr.GDR_ERR_NULL, gdr.GDR_OK
S, A, U, D, L, W = (gdr.GDR_ERR_SHAPE, gdr.GDR_ERR_ARG, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_ERR_DTYPE, gdr.GDR_ERR_ALIGN,
                    gdr.GDR_ERR_WORKSPACE)
NBYTES = 2 * 100 * 66


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), N), (dict(y=None), N), (dict(alpha=None), N), (dict(GATED, decay_a=None), N),
    (dict(GATED, decay_x=None), N), (dict(B=0), S), (dict(T=0), S), (dict(C=-1), S), (dict(C=(1 << 18) + 1), U),
    (dict(B=1 << 16, T=1 << 16), S), (dict(B=1, T=1 << 30, C=1024), S), (dict(io_dtype=2), D),
    (dict(decay_x=P(3)), A), (dict(decay_a=P(3)), A), (dict(gate_x=P(3)), A), (dict(normalise=1), A),
    (dict(GATED, normalise=2), A), (dict(reserved=1), A), (dict(x=P(0, 1)), L), (dict(alpha=P(1, 2)), L),
    (dict(y=P(2, 1)), L), (dict(h0=P(5, 2)), L), (dict(h_out=P(6, 1)), L), (dict(ckpt=P(7, 3)), L),
    (dict(workspace=P(30, 8)), L), (dict(y=P(0)), A), (dict(y=P(0, 2 * NBYTES - 2)), A),
    (dict(h0=P(5), h_out=P(5, 4)), A), (dict(ckpt=P(2, 64)), A), (dict(workspace=P(2, 1024)), A),
    (dict(h_out=P(6), ckpt=P(6)), A),
])
def test_scan_fwd_refusals(kw, status):
    assert gdr.call_channelwise("gdr_scan_fwd", _fwd(**kw)) == status


def _bwd(**kw):
    d = dict(B=2, T=100, C=66, io_dtype=gdr.GDR_BF16, x=P(0), alpha=P(1), grad_y=P(2), grad_x=P(8), grad_alpha=P(9),
             workspace=P(30), workspace_bytes=1 << 30)
    return gdr.ScanBwdArgs(**{**d, **kw})


GATED_B = dict(GATED, grad_alpha=None, grad_decay_x=P(10), grad_decay_a=P(11))


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), N), (dict(grad_y=None), N), (dict(grad_x=None), N), (dict(grad_alpha=None), N),
    (dict(GATED_B, grad_decay_x=None), N), (dict(GATED_B, grad_decay_a=None), N), (dict(GATED_B, gate_x=P(12)), N),
    (dict(GATED_B, grad_alpha=P(9)), A), (dict(grad_decay_x=P(9)), A), (dict(GATED_B, grad_gate_x=P(12)), A),
    (dict(grad_gate_x=P(12)), A), (dict(h0=P(13), ckpt=P(14)), A), (dict(T=0), S), (dict(io_dtype=-1), D),
    (dict(C=1 << 19), U), (dict(reserved=7), A), (dict(x_exp=P(15), x=P(0, 1), grad_y=P(2, 1)), L),
    (dict(grad_x=P(2)), A), (dict(grad_x=P(0, 64)), A), (dict(grad_h0=P(9)), A), (dict(x_exp=P(8)), A),
    (dict(workspace=None), W), (dict(workspace=None, workspace_bytes=0), W), (dict(workspace_bytes=16), W),
])
def test_scan_bwd_refusals(kw, status):
    assert gdr.call_channelwise("gdr_scan_bwd", _bwd(**kw)) == status


def test_workspace_queries():
    lib = gdr.load_library()
    assert lib.gdr_scan_bwd_workspace(ctypes.byref(_bwd())) > 0
    assert lib.gdr_scan_bwd_workspace(ctypes.byref(_bwd(x=None))) == 0
    assert lib.gdr_scan_fwd_workspace(ctypes.byref(_fwd(x=None))) == 0
    assert lib.gdr_scan_fwd_workspace(ctypes.byref(_fwd(T=1))) == 0        # one tile: no workspace
    assert lib.gdr_norm_bwd_workspace(ctypes.byref(_normb())) > 0
    assert lib.gdr_norm_bwd_workspace(ctypes.byref(_normb(grad_weight=None, grad_bias=None))) == 0
    for name in ("gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step", "gdr_norm_fwd", "gdr_norm_bwd", "gdr_ckpt8_pack",
                 "gdr_ckpt8_unpack"):
        assert getattr(lib, name)(None, None) == N


def _step(**kw):
    d = dict(N=4, C=66, io_dtype=gdr.GDR_F32, x=P(0), alpha=P(1), h=P(2), h_out=P(2), y=P(3))
    return gdr.ScanStepArgs(**{**d, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), N), (dict(h=None), N), (dict(h_out=None), N), (dict(y=None), N), (dict(alpha=None), N), (dict(N=0), S),
    (dict(N=1 << 14, C=1 << 17), S), (dict(io_dtype=5), D), (dict(normalise=1), A), (dict(gate_x=P(4)), A),
    (dict(h_out=P(2, 4)), A), (dict(y=P(2)), A), (dict(y=P(0)), A), (dict(h=P(2, 2)), L), (dict(y=P(3, 2)), L),
])
def test_scan_step_refusals(kw, status):
    assert gdr.call_channelwise("gdr_scan_step", _step(**kw)) == status


def _norm(**kw):
    d = dict(R=5, D=130, io_dtype=gdr.GDR_F32, eps=1e-5, x=P(0), y=P(1))
    return gdr.NormArgs(**{**d, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), N), (dict(y=None), N), (dict(x_code=P(2)), N), (dict(x_exp=P(2)), N), (dict(R=0), S), (dict(D=0), S),
    (dict(R=-3), S), (dict(R=1 << 31), S), (dict(D=65537), U), (dict(io_dtype=9), D), (dict(eps=-1.0), A),
    (dict(eps=float("nan")), A), (dict(eps=float("inf")), A), (dict(reserved=1), A), (dict(x=P(0, 2)), L),
    (dict(weight=P(3, 1)), L), (dict(mean=P(4, 2)), L), (dict(y=P(0)), A), (dict(mean=P(4), rstd=P(4, 16)), A),
    (dict(x_code=P(1, 8), x_exp=P(6)), A),
])
def test_norm_fwd_refusals(kw, status):
    assert gdr.call_channelwise("gdr_norm_fwd", _norm(**kw)) == status


def _normb(**kw):
    d = dict(R=5, D=130, io_dtype=gdr.GDR_BF16, x=P(0), mean=P(1), rstd=P(2), grad_y=P(3), grad_x=P(4), grad_weight=P(5),
             grad_bias=P(6), workspace=P(30), workspace_bytes=1 << 30)
    return gdr.NormBwdArgs(**{**d, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), N), (dict(mean=None), N), (dict(rstd=None), N), (dict(grad_y=None), N), (dict(grad_x=None), N),
    (dict(R=0), S), (dict(D=65537), U), (dict(io_dtype=3), D), (dict(grad_x=P(3)), A), (dict(grad_x=P(0)), A),
    (dict(grad_bias=P(5)), A), (dict(grad_y=P(3, 1)), L), (dict(workspace=P(30, 4)), L), (dict(workspace=None), W),
    (dict(workspace_bytes=32), W),
])
def test_norm_bwd_refusals(kw, status):
    assert gdr.call_channelwise("gdr_norm_bwd", _normb(**kw)) == status


@pytest.mark.parametrize("name,cls,out", [("gdr_ckpt8_pack", gdr.Ckpt8PackArgs, "code"),
                                          ("gdr_ckpt8_unpack", gdr.Ckpt8UnpackArgs, "x")])
def test_ckpt8_refusals(name, cls, out):
    d = dict(R=5, D=130, io_dtype=gdr.GDR_F32, x=P(0), code=P(1), exp=P(2))
    for kw, status in [(dict(x=None), N), (dict(code=None), N), (dict(exp=None), N), (dict(R=0), S), (dict(D=-1), S),
                       (dict(io_dtype=4), D), (dict(D=(1 << 30) + 1), U), (dict(R=1 << 31), S), (dict(x=P(0, 2)), L),
                       ({out: P(2)}, A), (dict(code=P(0, 100)), A)]:
        assert gdr.call_channelwise(name, cls(**{**d, **kw})) == status, (name, kw)


def test_binding_checks():
    """Shapes, types and contiguity are refused by name before the device is looked at;
    good arguments on the CPU get as far as the device."""
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    x, al, A, h = torch.zeros(2, 5, 8, dtype=bf), torch.ones(2, 5, 8), torch.ones(8), torch.zeros(2, 8)
    calls = [
        ("GPU", lambda: gdr.gdr_scan_fwd(x, al, h0=h)),
        ("GPU", lambda: gdr.gdr_scan_fwd_gated(x, x, A, gate_x=x)),
        ("GPU", lambda: gdr.gdr_scan_bwd(x, al, x)),
        ("GPU", lambda: gdr.gdr_scan_step(h, x[:, 0].contiguous(), al[:, 0].contiguous())),
        ("GPU", lambda: gdr.gdr_norm_fwd(x, A, A)),
        ("GPU", lambda: gdr.gdr_norm_bwd(x, x, al[..., 0].contiguous(), al[..., 0].contiguous(), A)),
        ("GPU", lambda: gdr.gdr_ckpt8_pack(x)),
        ("B,T,C", lambda: gdr.gdr_scan_fwd(x[0], al)),
        ("alpha", lambda: gdr.gdr_scan_fwd(x, None)),
        ("alpha", lambda: gdr.gdr_scan_fwd(x, al.to(bf))),
        ("alpha", lambda: gdr.gdr_scan_bwd(x, al[:, :4].contiguous(), x)),
        ("contiguous", lambda: gdr.gdr_scan_fwd(x.transpose(0, 1), al.transpose(0, 1).contiguous())),
        ("decay_x", lambda: gdr.gdr_scan_fwd_gated(x, x.float(), A)),
        ("decay_a", lambda: gdr.gdr_scan_fwd_gated(x, x, None)),
        ("decay_a", lambda: gdr.gdr_scan_step_gated(h, x[:, 0].contiguous(), x[:, 0].contiguous(), A[:4])),
        ("gate_x", lambda: gdr.gdr_scan_fwd_gated(x, x, A, gate_x=x[:1])),
        ("h0", lambda: gdr.gdr_scan_fwd(x, al, h0=h.to(bf))),
        ("not both", lambda: gdr.gdr_scan_bwd(x, al, x, h0=h, ckpt=torch.zeros(2, 1, 8))),
        ("ckpt", lambda: gdr.gdr_scan_bwd(x, al, x, ckpt=torch.zeros(2, 2, 8))),
        ("grad_h", lambda: gdr.gdr_scan_bwd(x, al, x, grad_h=h[:1])),
        (r"x\[0\]", lambda: gdr.gdr_scan_bwd((x, h), al, x)),
        ("N,C", lambda: gdr.gdr_scan_step(h, x, al)),
        ("bfloat16 or float32", lambda: gdr.gdr_scan_fwd(x.half(), al)),
        ("weight", lambda: gdr.gdr_norm_fwd(x, A[:7])),
        ("bias", lambda: gdr.gdr_norm_fwd(x, A, A.to(bf))),
        ("contiguous", lambda: gdr.gdr_norm_fwd(x[..., ::2])),
        ("mean", lambda: gdr.gdr_norm_bwd(x, x, A, A)),
        ("mean", lambda: gdr.gdr_norm_bwd(x, x, None, A)),
        ("x has shape", lambda: gdr.gdr_norm_bwd(x, x[0], al[..., 0], al[..., 0])),
        ("code", lambda: gdr.gdr_ckpt8_unpack(x, x)),
        ("D", lambda: gdr.gdr_ckpt8_pack(torch.zeros(()))),
        ("bfloat16 or float32", lambda: gdr.gdr_norm_fwd(x.double())),
    ]
    for match, call in calls:
        with pytest.raises(ValueError, match=match):
            call()


def test_host_half_under_sanitizers(tmp_path):
    import shutil
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "harness"
    csrc = os.path.join(ROOT, "recurrent_state_memory_amd", "csrc")
    cmd = [gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
           "-I" + csrc, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g",
           os.path.join(ROOT, "tests", "channelwise_host_harness.cpp"), os.path.join(csrc, "scan_api.cpp"),
           os.path.join(csrc, "norm_api.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "sanitizer" in r.stderr.lower():
        pytest.skip("sanitizer runtime not available: " + r.stderr[-200:])
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1:verify_asan_link_order=0")
    out = subprocess.run([str(exe)], capture_output=True, text=True, env=env)
    assert out.returncode == 0 and "CHANNELWISE_HARNESS_OK" in out.stdout, out.stdout + out.stderr
