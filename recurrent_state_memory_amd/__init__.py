"""MI355X (gfx950) gated delta-rule library: Python binding over libgdr.so.

The binding only marshals arguments: it reads device pointers and the
current HIP stream from torch tensors, fills the C structs declared in
``include/gdr.h`` and calls the exported functions.  Every step of the
computation runs in the HIP kernels of ``libgdr.so``; there is no fallback.
If the library has not been built, every call raises ``RuntimeError``.

Entry points (same names as the C ABI):

* ``gdr_chunk_fwd``   -- chunked forward over a sequence, returns (o, S_out)
* ``gdr_chunk_fwd_gated`` -- the same with the decay activation (and optionally
  the q/k L2 normalisation) computed in the kernel from raw inputs
* ``gdr_chunk_bwd``   -- gradients of the plain-erase forward (recomputes it)
* ``gdr_step_decode`` -- one token on a batch of states, in place, returns o
* ``gdr_raven_fwd``   -- the Raven routing slot memory (include/gdr_raven.h),
  returns (o, Sk_out, Sv_out)
* ``gdr_perm_fwd``    -- the delta rule with partial-permutation transitions
  (include/gdr_perm.h), returns (o, S_out)
* ``gdr_scan_fwd``, ``gdr_scan_bwd``, ``gdr_scan_step`` and their ``_gated``
  forms -- the channelwise gated linear recurrence (include/gdr_scan.h)
* ``gdr_norm_fwd``, ``gdr_norm_bwd`` -- layer norm (include/gdr_norm.h)
* ``gdr_ckpt8_pack``, ``gdr_ckpt8_unpack`` -- activations kept in 8 bits for the
  backward (include/gdr_ckpt8.h)
* ``gdr_conv_fwd``, ``gdr_conv_bwd``, ``gdr_conv_step`` -- short causal convolution
  (include/gdr_conv.h)
* ``gdr_ssm_fwd``, ``gdr_ssm_bwd``, ``gdr_ssm_step`` -- selective state space scan
  (include/gdr_ssm.h)
* ``gdr_gnorm_fwd``, ``gdr_gnorm_bwd`` -- group norm with its activation or gate
  (include/gdr_gnorm.h)

The channelwise operators (the last six lines) run on the device of their
tensors, on its current stream or on ``stream``, and allocate what they return
and their workspaces on that stream.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

GDR_OK, GDR_ERR_NULL, GDR_ERR_SHAPE, GDR_ERR_DTYPE, GDR_ERR_UNSUPPORTED, \
    GDR_ERR_ALIGN, GDR_ERR_WORKSPACE, GDR_ERR_HIP, GDR_ERR_ARG = range(9)
GDR_F32, GDR_BF16 = 0, 1
GDR_DECAY_DIAG, GDR_DECAY_ROT2, GDR_DECAY_DIHEDRAL = 0, 1, 2
ABI_VERSION = 1

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32


class FwdArgs(ctypes.Structure):
    """Mirror of ``gdr_fwd_args``."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("H", _i32), ("dk", _i32), ("dv", _i32),
        ("chunk", _i32), ("io_dtype", _i32), ("decay", _i32),
        ("q", _vp), ("k", _vp), ("v", _vp), ("alpha", _vp), ("theta", _vp),
        ("beta", _vp), ("w", _vp), ("beta_logit", _vp), ("ub_down", _vp),
        ("ub_up", _vp), ("ub_rank", _i32), ("reserved0", _i32), ("m_carry", _vp),
        ("S0", _vp), ("o", _vp), ("S_out", _vp), ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class GateArgs(ctypes.Structure):
    """Mirror of ``gdr_gate_args``."""
    _fields_ = [("decay_x", _vp), ("decay_a", _vp), ("qk_l2norm", _i32), ("reserved", _i32)]


class GateGrads(ctypes.Structure):
    """Mirror of ``gdr_gate_grads``."""
    _fields_ = [("grad_decay_x", _vp), ("grad_decay_a", _vp)]


class BwdArgs(ctypes.Structure):
    """Mirror of ``gdr_bwd_args``."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("H", _i32), ("dk", _i32), ("dv", _i32), ("decay", _i32),
        ("q", _vp), ("k", _vp), ("v", _vp), ("alpha", _vp), ("theta", _vp),
        ("beta", _vp), ("w", _vp), ("S0", _vp), ("grad_o", _vp), ("grad_S", _vp),
        ("grad_q", _vp), ("grad_k", _vp), ("grad_v", _vp), ("grad_alpha", _vp),
        ("grad_theta", _vp), ("grad_beta", _vp), ("grad_w", _vp), ("grad_S0", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class StepArgs(ctypes.Structure):
    """Mirror of ``gdr_step_args``."""
    _fields_ = [
        ("N", _i32), ("H", _i32), ("dk", _i32), ("dv", _i32),
        ("io_dtype", _i32), ("decay", _i32),
        ("q", _vp), ("k", _vp), ("v", _vp), ("alpha", _vp), ("theta", _vp),
        ("beta", _vp), ("w", _vp), ("S", _vp), ("o", _vp),
    ]


class RavenArgs(ctypes.Structure):
    """Mirror of ``gdr_raven_args`` (include/gdr_raven.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("H", _i32), ("dk", _i32), ("dv", _i32),
        ("slots", _i32), ("topk", _i32), ("scale", ctypes.c_float),
        ("q", _vp), ("k", _vp), ("v", _vp), ("z", _vp), ("a", _vp),
        ("Sk0", _vp), ("Sv0", _vp), ("o", _vp), ("Sk_out", _vp), ("Sv_out", _vp),
    ]


class PermArgs(ctypes.Structure):
    """Mirror of ``gdr_perm_args`` (include/gdr_perm.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("H", _i32), ("dk", _i32), ("dv", _i32),
        ("q", _vp), ("k", _vp), ("v", _vp), ("src", _vp), ("beta", _vp), ("w", _vp),
        ("S0", _vp), ("o", _vp), ("S_out", _vp),
    ]


class GdrError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"gdr status {status}: {msg}")
        self.status = status


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libgdr.so (built by ``python -m recurrent_state_memory_amd.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with `python -m recurrent_state_memory_amd.build`")
    lib = ctypes.CDLL(p)
    lib.gdr_chunk_fwd.argtypes = [ctypes.POINTER(FwdArgs), _vp]
    lib.gdr_chunk_fwd.restype = ctypes.c_int
    lib.gdr_chunk_fwd_gated.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(GateArgs), _vp]
    lib.gdr_chunk_fwd_gated.restype = ctypes.c_int
    lib.gdr_chunk_bwd.argtypes = [ctypes.POINTER(BwdArgs), _vp]
    lib.gdr_chunk_bwd.restype = ctypes.c_int
    lib.gdr_chunk_bwd_noalloc.argtypes = [ctypes.POINTER(BwdArgs), _vp]
    lib.gdr_chunk_bwd_noalloc.restype = ctypes.c_int
    lib.gdr_chunk_bwd_gated.argtypes = [ctypes.POINTER(BwdArgs), ctypes.POINTER(GateArgs),
                                        ctypes.POINTER(GateGrads), _vp]
    lib.gdr_chunk_bwd_gated.restype = ctypes.c_int
    lib.gdr_chunk_bwd_gated_workspace.argtypes = [ctypes.POINTER(BwdArgs), ctypes.POINTER(GateArgs)]
    lib.gdr_chunk_bwd_gated_workspace.restype = ctypes.c_size_t
    lib.gdr_chunk_bwd_workspace.argtypes = [ctypes.POINTER(BwdArgs)]
    lib.gdr_chunk_bwd_workspace.restype = ctypes.c_size_t
    lib.gdr_chunk_fwd_workspace.argtypes = [ctypes.POINTER(FwdArgs)]
    lib.gdr_chunk_fwd_workspace.restype = ctypes.c_size_t
    lib.gdr_step_decode.argtypes = [ctypes.POINTER(StepArgs), _vp]
    lib.gdr_step_decode.restype = ctypes.c_int
    lib.gdr_raven_fwd.argtypes = [ctypes.POINTER(RavenArgs), _vp]
    lib.gdr_raven_fwd.restype = ctypes.c_int
    lib.gdr_perm_fwd.argtypes = [ctypes.POINTER(PermArgs), _vp]
    lib.gdr_perm_fwd.restype = ctypes.c_int
    for name, struct in _CHANNELWISE.items():
        getattr(lib, name).argtypes = [ctypes.POINTER(struct), _vp]
        getattr(lib, name).restype = ctypes.c_int
    for name, struct in _CHANNELWISE_WS.items():
        getattr(lib, name).argtypes = [ctypes.POINTER(struct)]
        getattr(lib, name).restype = ctypes.c_size_t
    lib.gdr_status_str.argtypes = [ctypes.c_int]
    lib.gdr_status_str.restype = ctypes.c_char_p
    lib.gdr_abi_version.argtypes = []
    lib.gdr_abi_version.restype = ctypes.c_int
    if lib.gdr_abi_version() != ABI_VERSION:
        raise RuntimeError("libgdr ABI version mismatch")
    if path is None:
        _lib = lib
    return lib


def status_str(status: int) -> str:
    return load_library().gdr_status_str(status).decode()


def _check(status: int):
    if status != GDR_OK:
        raise GdrError(status, status_str(status))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gdr: tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("gdr: tensors must be contiguous")
    return t.data_ptr()


def _expect(t, name: str, shape, dtype, required: bool = True):
    """Check one argument's presence, shape and dtype (before any pointer is taken,
    so that a wrong shape can never make a kernel read past an allocation)."""
    if t is None:
        if required:
            raise ValueError(f"gdr: {name} is required")
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"gdr: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"gdr: {name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"gdr: {name} must be contiguous")


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _io(t):
    import torch
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    if t.dtype == torch.float32:
        return GDR_F32
    raise ValueError(f"gdr: q/k/v must be bfloat16 or float32, got {t.dtype}")


def call_chunk_fwd(args: FwdArgs, stream=None) -> int:
    """Raw call with a filled ``FwdArgs``; returns the status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_chunk_fwd(ctypes.byref(args), s)


def call_chunk_fwd_gated(args: FwdArgs, gate: GateArgs, stream=None) -> int:
    """Raw call with filled ``FwdArgs`` and ``GateArgs``; returns the status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_chunk_fwd_gated(ctypes.byref(args), ctypes.byref(gate), s)


def call_chunk_bwd(args: BwdArgs, stream=None) -> int:
    """Raw call with a filled ``BwdArgs``; returns the status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_chunk_bwd(ctypes.byref(args), s)


def call_chunk_bwd_gated(args: BwdArgs, gate: GateArgs, grads: GateGrads, stream=None) -> int:
    """Raw call with filled ``BwdArgs``, ``GateArgs`` and ``GateGrads``; returns the
    status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_chunk_bwd_gated(ctypes.byref(args), ctypes.byref(gate), ctypes.byref(grads), s)


def call_chunk_bwd_noalloc(args: BwdArgs, stream=None) -> int:
    """Raw call of the static-scratch backward (``args.workspace`` must be
    NULL); returns the status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_chunk_bwd_noalloc(ctypes.byref(args), s)


def call_raven_fwd(args: RavenArgs, stream=None) -> int:
    """Raw call with a filled ``RavenArgs``; returns the status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_raven_fwd(ctypes.byref(args), s)


def call_perm_fwd(args: PermArgs, stream=None) -> int:
    """Raw call with a filled ``PermArgs``; returns the status code."""
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_perm_fwd(ctypes.byref(args), s)


def call_step_decode(args: StepArgs, stream=None) -> int:
    lib = load_library()
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return lib.gdr_step_decode(ctypes.byref(args), s)


def _decay_kind(rot, reflections):
    if reflections and not rot:
        raise ValueError("gdr: reflection blocks need theta (2x2 blocks)")
    if reflections:
        return GDR_DECAY_DIHEDRAL
    return GDR_DECAY_ROT2 if rot else GDR_DECAY_DIAG


def gdr_chunk_fwd(q, k, v, alpha, w, beta=None, *, theta=None, S0=None, chunk=64,
                  o=None, S_out=None, return_state=True, beta_logit=None,
                  ub_down=None, ub_up=None, m_carry=None, reflections=False, stream=None):
    """Chunked gated delta-rule forward (see ``gdr_chunk_fwd`` in include/gdr.h).

    q, k [B,T,H,dk], v [B,T,H,dv] (bf16 or fp32, same dtype); alpha fp32
    [B,T,H,dk] (per-channel decay) or [B,T,H,dk/2] with ``theta`` (2x2
    rotation-decay blocks); beta, w fp32 [B,T,H].  ``reflections=True`` (with
    ``theta``) makes a block whose alpha is negative (sign bit set) the
    reflection of magnitude |alpha| (GDR_DECAY_DIHEDRAL).  Content-aware erase: pass
    ``beta_logit``, ``ub_down`` [H,r,dv], ``ub_up`` [H,r] instead of ``beta``.
    Returns (o [B,T,H,dv], S_out [B,H,dv,dk] fp32 or None).

    Every tensor's shape, dtype and contiguity is checked against (B, T, H,
    dk, dv) before anything reaches the library.
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("gdr: q, k and v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    io = q.dtype
    f32 = torch.float32
    _io(q)
    _expect(k, "k", (B, T, H, dk), io)
    _expect(v, "v", (B, T, H, dv), io)
    rot = theta is not None
    content = beta_logit is not None
    gshape = (B, T, H, dk // 2) if rot else (B, T, H, dk)
    if rot and dk % 2:
        raise ValueError("gdr: rotation-decay blocks need an even d_k")
    _expect(alpha, "alpha", gshape, f32)
    _expect(theta, "theta", gshape, f32, required=False)
    _expect(w, "w", (B, T, H), f32)
    if content:
        if beta is not None:
            raise ValueError("gdr: pass either beta or beta_logit, not both")
        if ub_down is None or ub_up is None or ub_up.dim() != 2:
            raise ValueError("gdr: the content-aware erase needs ub_down [H,r,dv] and ub_up [H,r]")
        r = ub_up.shape[-1]
        _expect(beta_logit, "beta_logit", (B, T, H), f32)
        _expect(ub_down, "ub_down", (H, r, dv), f32)
        _expect(ub_up, "ub_up", (H, r), f32)
        _expect(m_carry, "m_carry", (B, H, dv), f32, required=False)
    else:
        if ub_down is not None or ub_up is not None or m_carry is not None:
            raise ValueError("gdr: ub_down, ub_up and m_carry belong to the content-aware erase")
        _expect(beta, "beta", (B, T, H), f32)
    _expect(S0, "S0", (B, H, dv, dk), f32, required=False)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=io, device=q.device)
    _expect(o, "o", (B, T, H, dv), io)
    if S_out is None and return_state:
        S_out = torch.empty((B, H, dv, dk), dtype=f32, device=q.device)
    _expect(S_out, "S_out", (B, H, dv, dk), f32, required=False)
    a = FwdArgs()
    a.B, a.T, a.H, a.dk, a.dv, a.chunk = B, T, H, dk, dv, chunk
    a.io_dtype = _io(q)
    a.decay = _decay_kind(rot, reflections)
    a.q, a.k, a.v, a.alpha, a.theta = map(_ptr, (q, k, v, alpha, theta))
    a.beta, a.w, a.beta_logit = map(_ptr, (beta, w, beta_logit))
    a.ub_down, a.ub_up, a.m_carry = map(_ptr, (ub_down, ub_up, m_carry))
    a.ub_rank = 0 if ub_up is None else int(ub_up.shape[-1])
    a.S0, a.o, a.S_out = _ptr(S0), _ptr(o), _ptr(S_out)
    a.workspace, a.workspace_bytes = None, 0
    _check(call_chunk_fwd(a, _stream(stream)))
    return o, S_out


def gdr_chunk_fwd_gated(q, k, v, decay_x, decay_a, w, beta, *, theta=None, qk_l2norm=True,
                        S0=None, chunk=64, o=None, S_out=None, return_state=True, stream=None):
    """Forward with the decay activation in the kernel (``gdr_chunk_fwd_gated`` in
    include/gdr.h): decay = exp(-decay_a[h] * softplus(decay_x)).

    q, k [B,T,H,dk], v [B,T,H,dv] bf16 (raw q, k when ``qk_l2norm``); decay_x
    bf16 [B,T,H,dk] (per-channel decay) or [B,T,H,dk/2] with ``theta`` fp32 of
    the same shape (2x2 rotation-decay blocks); decay_a fp32 [H]; beta, w fp32
    [B,T,H].  Returns (o [B,T,H,dv] bf16, S_out [B,H,dv,dk] fp32 or None).
    Shapes, dtypes and contiguity are checked first.
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("gdr: q, k and v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    bf, f32 = torch.bfloat16, torch.float32
    _expect(q, "q", (B, T, H, dk), bf)
    _expect(k, "k", (B, T, H, dk), bf)
    _expect(v, "v", (B, T, H, dv), bf)
    rot = theta is not None
    if rot and dk % 2:
        raise ValueError("gdr: rotation-decay blocks need an even d_k")
    gshape = (B, T, H, dk // 2) if rot else (B, T, H, dk)
    _expect(decay_x, "decay_x", gshape, bf)
    _expect(theta, "theta", gshape, f32, required=False)
    _expect(decay_a, "decay_a", (H,), f32)
    _expect(w, "w", (B, T, H), f32)
    _expect(beta, "beta", (B, T, H), f32)
    _expect(S0, "S0", (B, H, dv, dk), f32, required=False)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=bf, device=q.device)
    _expect(o, "o", (B, T, H, dv), bf)
    if S_out is None and return_state:
        S_out = torch.empty((B, H, dv, dk), dtype=f32, device=q.device)
    _expect(S_out, "S_out", (B, H, dv, dk), f32, required=False)
    a = FwdArgs()
    a.B, a.T, a.H, a.dk, a.dv, a.chunk = B, T, H, dk, dv, chunk
    a.io_dtype = GDR_BF16
    a.decay = GDR_DECAY_ROT2 if rot else GDR_DECAY_DIAG
    a.q, a.k, a.v, a.theta = map(_ptr, (q, k, v, theta))
    a.alpha = None
    a.beta, a.w = _ptr(beta), _ptr(w)
    a.beta_logit = a.ub_down = a.ub_up = a.m_carry = None
    a.ub_rank = 0
    a.S0, a.o, a.S_out = _ptr(S0), _ptr(o), _ptr(S_out)
    a.workspace, a.workspace_bytes = None, 0
    g = GateArgs()
    g.decay_x, g.decay_a = _ptr(decay_x), _ptr(decay_a)
    g.qk_l2norm, g.reserved = int(bool(qk_l2norm)), 0
    _check(call_chunk_fwd_gated(a, g, _stream(stream)))
    return o, S_out


def gdr_chunk_bwd(q, k, v, alpha, w, beta, grad_o, *, theta=None, S0=None, grad_S=None,
                  need_grad_S0=True, workspace=None, stream=None):
    """Gradients of the plain-erase forward (``gdr_chunk_bwd`` in include/gdr.h).

    Inputs as ``gdr_chunk_fwd`` (bf16 q, k, v; fp32 alpha [and theta], beta,
    w; optional S0) plus grad_o [B,T,H,dv] bf16 and optional grad_S
    [B,H,dv,dk] fp32.  Returns a dict of fp32 tensors: q, k, v, alpha, beta,
    w, theta (rotation decay only) and S0 (when ``need_grad_S0``).  The
    workspace (``gdr_chunk_bwd_workspace`` bytes) is allocated here unless a
    large enough uint8 CUDA tensor is passed.
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("gdr: q, k and v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    bf, f32 = torch.bfloat16, torch.float32
    _expect(q, "q", (B, T, H, dk), bf)
    _expect(k, "k", (B, T, H, dk), bf)
    _expect(v, "v", (B, T, H, dv), bf)
    rot = theta is not None
    if rot and dk % 2:
        raise ValueError("gdr: rotation-decay blocks need an even d_k")
    gshape = (B, T, H, dk // 2) if rot else (B, T, H, dk)
    _expect(alpha, "alpha", gshape, f32)
    _expect(theta, "theta", gshape, f32, required=False)
    _expect(w, "w", (B, T, H), f32)
    _expect(beta, "beta", (B, T, H), f32)
    _expect(S0, "S0", (B, H, dv, dk), f32, required=False)
    _expect(grad_o, "grad_o", (B, T, H, dv), bf)
    _expect(grad_S, "grad_S", (B, H, dv, dk), f32, required=False)
    dev = q.device
    g = {"q": torch.empty((B, T, H, dk), dtype=f32, device=dev),
         "k": torch.empty((B, T, H, dk), dtype=f32, device=dev),
         "v": torch.empty((B, T, H, dv), dtype=f32, device=dev),
         "alpha": torch.empty(gshape, dtype=f32, device=dev),
         "beta": torch.empty((B, T, H), dtype=f32, device=dev),
         "w": torch.empty((B, T, H), dtype=f32, device=dev)}
    if rot:
        g["theta"] = torch.empty(gshape, dtype=f32, device=dev)
    if need_grad_S0:
        g["S0"] = torch.empty((B, H, dv, dk), dtype=f32, device=dev)
    a = BwdArgs()
    a.B, a.T, a.H, a.dk, a.dv = B, T, H, dk, dv
    a.decay = GDR_DECAY_ROT2 if rot else GDR_DECAY_DIAG
    a.q, a.k, a.v, a.alpha, a.theta = map(_ptr, (q, k, v, alpha, theta))
    a.beta, a.w, a.S0, a.grad_o, a.grad_S = map(_ptr, (beta, w, S0, grad_o, grad_S))
    a.grad_q, a.grad_k, a.grad_v = _ptr(g["q"]), _ptr(g["k"]), _ptr(g["v"])
    a.grad_alpha, a.grad_theta = _ptr(g["alpha"]), _ptr(g.get("theta"))
    a.grad_beta, a.grad_w, a.grad_S0 = _ptr(g["beta"]), _ptr(g["w"]), _ptr(g.get("S0"))
    need = load_library().gdr_chunk_bwd_workspace(ctypes.byref(a))
    if need == 0:
        _check(call_chunk_bwd(a, _stream(stream)))   # reports why the arguments are invalid
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"gdr: workspace must be a uint8 tensor of at least {need} bytes")
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    _check(call_chunk_bwd(a, _stream(stream)))
    return g


def gdr_chunk_bwd_gated(q, k, v, decay_x, decay_a, w, beta, grad_o, *, theta=None,
                        qk_l2norm=True, S0=None, grad_S=None, need_grad_S0=True,
                        workspace=None, stream=None):
    """Gradients of the gated forward (``gdr_chunk_bwd_gated`` in include/gdr.h).

    Inputs as ``gdr_chunk_fwd_gated`` (bf16 q, k, v, raw q and k when
    ``qk_l2norm``; bf16 decay_x [B,T,H,dk] or [B,T,H,dk/2] with ``theta``; fp32
    decay_a [H], beta, w) plus grad_o [B,T,H,dv] bf16 and optional grad_S
    [B,H,dv,dk] fp32.  Returns a dict of fp32 tensors: q, k (of the raw
    inputs), v, x (decay_x), a (decay_a), beta, w, theta (rotation decay only)
    and S0 (when ``need_grad_S0``).  The workspace
    (``gdr_chunk_bwd_gated_workspace`` bytes) is allocated here unless a large
    enough uint8 CUDA tensor is passed.
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("gdr: q, k and v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    bf, f32 = torch.bfloat16, torch.float32
    _expect(q, "q", (B, T, H, dk), bf)
    _expect(k, "k", (B, T, H, dk), bf)
    _expect(v, "v", (B, T, H, dv), bf)
    rot = theta is not None
    if rot and dk % 2:
        raise ValueError("gdr: rotation-decay blocks need an even d_k")
    gshape = (B, T, H, dk // 2) if rot else (B, T, H, dk)
    _expect(decay_x, "decay_x", gshape, bf)
    _expect(theta, "theta", gshape, f32, required=False)
    _expect(decay_a, "decay_a", (H,), f32)
    _expect(w, "w", (B, T, H), f32)
    _expect(beta, "beta", (B, T, H), f32)
    _expect(S0, "S0", (B, H, dv, dk), f32, required=False)
    _expect(grad_o, "grad_o", (B, T, H, dv), bf)
    _expect(grad_S, "grad_S", (B, H, dv, dk), f32, required=False)
    dev = q.device
    g = {"q": torch.empty((B, T, H, dk), dtype=f32, device=dev),
         "k": torch.empty((B, T, H, dk), dtype=f32, device=dev),
         "v": torch.empty((B, T, H, dv), dtype=f32, device=dev),
         "x": torch.empty(gshape, dtype=f32, device=dev),
         "a": torch.empty((H,), dtype=f32, device=dev),
         "beta": torch.empty((B, T, H), dtype=f32, device=dev),
         "w": torch.empty((B, T, H), dtype=f32, device=dev)}
    if rot:
        g["theta"] = torch.empty(gshape, dtype=f32, device=dev)
    if need_grad_S0:
        g["S0"] = torch.empty((B, H, dv, dk), dtype=f32, device=dev)
    a = BwdArgs()
    a.B, a.T, a.H, a.dk, a.dv = B, T, H, dk, dv
    a.decay = GDR_DECAY_ROT2 if rot else GDR_DECAY_DIAG
    a.q, a.k, a.v, a.theta = map(_ptr, (q, k, v, theta))
    a.alpha, a.grad_alpha = None, None
    a.beta, a.w, a.S0, a.grad_o, a.grad_S = map(_ptr, (beta, w, S0, grad_o, grad_S))
    a.grad_q, a.grad_k, a.grad_v = _ptr(g["q"]), _ptr(g["k"]), _ptr(g["v"])
    a.grad_theta = _ptr(g.get("theta"))
    a.grad_beta, a.grad_w, a.grad_S0 = _ptr(g["beta"]), _ptr(g["w"]), _ptr(g.get("S0"))
    ga = GateArgs()
    ga.decay_x, ga.decay_a = _ptr(decay_x), _ptr(decay_a)
    ga.qk_l2norm, ga.reserved = int(bool(qk_l2norm)), 0
    gg = GateGrads()
    gg.grad_decay_x, gg.grad_decay_a = _ptr(g["x"]), _ptr(g["a"])
    need = load_library().gdr_chunk_bwd_gated_workspace(ctypes.byref(a), ctypes.byref(ga))
    if need == 0:
        _check(call_chunk_bwd_gated(a, ga, gg, _stream(stream)))   # reports why the arguments are invalid
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"gdr: workspace must be a uint8 tensor of at least {need} bytes")
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    _check(call_chunk_bwd_gated(a, ga, gg, _stream(stream)))
    return g


def gdr_step_decode(S, q, k, v, alpha, beta, w, *, theta=None, o=None, reflections=False,
                    stream=None):
    """One token on N states in place (see ``gdr_step_decode`` in include/gdr.h).

    S [N,H,dv,dk] fp32 (overwritten), q,k [N,H,dk], v [N,H,dv], alpha [N,H,dk]
    or gamma [N,H,dk/2] with theta, beta, w [N,H]; ``reflections`` as in
    ``gdr_chunk_fwd``.  Returns o [N,H,dv].
    Every tensor's shape, dtype and contiguity is checked first.
    """
    import torch
    if S.dim() != 4:
        raise ValueError("gdr: S must be [N,H,dv,dk]")
    N, H, dv, dk = S.shape
    f32 = torch.float32
    io = q.dtype
    _io(q)
    _expect(S, "S", (N, H, dv, dk), f32)
    _expect(q, "q", (N, H, dk), io)
    _expect(k, "k", (N, H, dk), io)
    _expect(v, "v", (N, H, dv), io)
    rot = theta is not None
    gshape = (N, H, dk // 2) if rot else (N, H, dk)
    _expect(alpha, "alpha", gshape, f32)
    _expect(theta, "theta", gshape, f32, required=False)
    _expect(beta, "beta", (N, H), f32)
    _expect(w, "w", (N, H), f32)
    if o is None:
        o = torch.empty((N, H, dv), dtype=io, device=q.device)
    _expect(o, "o", (N, H, dv), io)
    a = StepArgs()
    a.N, a.H, a.dk, a.dv = N, H, dk, dv
    a.io_dtype = _io(q)
    a.decay = _decay_kind(rot, reflections)
    a.q, a.k, a.v, a.alpha, a.theta = map(_ptr, (q, k, v, alpha, theta))
    a.beta, a.w, a.S, a.o = map(_ptr, (beta, w, S, o))
    _check(call_step_decode(a, _stream(stream)))
    return o


def gdr_raven_fwd(q, k, v, z, a, *, topk, scale=None, Sk0=None, Sv0=None, o=None,
                  Sk_out=None, Sv_out=None, return_state=True, stream=None):
    """Raven routing slot-memory forward (see ``gdr_raven_fwd`` in
    include/gdr_raven.h).

    q, k [B,T,H,dk], v [B,T,H,dv], router logits z [B,T,H,slots], all bf16;
    decay rate a fp32 [B,T,H] (finite, <= 0); ``topk`` slots written per token;
    ``scale`` of the read-out logits (default 1/sqrt(dk)); start slots Sk0
    [B,H,slots,dk], Sv0 [B,H,slots,dv] fp32 or None (zero).  Returns
    (o [B,T,H,dv] bf16, Sk_out, Sv_out) -- the states None unless
    ``return_state`` or given.
    """
    import math
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or z.dim() != 4:
        raise ValueError("gdr: q, k, v and z must be [B,T,H,*]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    M = z.shape[-1]
    bf, f32 = torch.bfloat16, torch.float32
    _expect(q, "q", (B, T, H, dk), bf)
    _expect(k, "k", (B, T, H, dk), bf)
    _expect(v, "v", (B, T, H, dv), bf)
    _expect(z, "z", (B, T, H, M), bf)
    _expect(a, "a", (B, T, H), f32)
    _expect(Sk0, "Sk0", (B, H, M, dk), f32, required=False)
    _expect(Sv0, "Sv0", (B, H, M, dv), f32, required=False)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=bf, device=q.device)
    _expect(o, "o", (B, T, H, dv), bf)
    if return_state:
        if Sk_out is None:
            Sk_out = torch.empty((B, H, M, dk), dtype=f32, device=q.device)
        if Sv_out is None:
            Sv_out = torch.empty((B, H, M, dv), dtype=f32, device=q.device)
    _expect(Sk_out, "Sk_out", (B, H, M, dk), f32, required=False)
    _expect(Sv_out, "Sv_out", (B, H, M, dv), f32, required=False)
    r = RavenArgs()
    r.B, r.T, r.H, r.dk, r.dv, r.slots, r.topk = B, T, H, dk, dv, M, int(topk)
    r.scale = 1.0 / math.sqrt(dk) if scale is None else float(scale)
    r.q, r.k, r.v, r.z, r.a = map(_ptr, (q, k, v, z, a))
    r.Sk0, r.Sv0, r.o, r.Sk_out, r.Sv_out = map(_ptr, (Sk0, Sv0, o, Sk_out, Sv_out))
    _check(call_raven_fwd(r, _stream(stream)))
    return o, Sk_out, Sv_out


def gdr_perm_fwd(q, k, v, w, src, beta, *, S0=None, o=None, S_out=None, return_state=True,
                 stream=None):
    """Delta rule with partial-permutation transitions (see ``gdr_perm_fwd`` in
    include/gdr_perm.h): column j of S D_t is column src[j] of S (zero for a
    value outside [0, dk)).

    q, k [B,T,H,dk], v [B,T,H,dv] bf16; w, beta fp32 [B,T,H]; src int16
    [B,T,H,dk]; S0 fp32 [B,H,dv,dk] or None.  Returns (o [B,T,H,dv] bf16, S_out).
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("gdr: q, k and v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    bf, f32 = torch.bfloat16, torch.float32
    _expect(q, "q", (B, T, H, dk), bf)
    _expect(k, "k", (B, T, H, dk), bf)
    _expect(v, "v", (B, T, H, dv), bf)
    _expect(src, "src", (B, T, H, dk), torch.int16)
    _expect(w, "w", (B, T, H), f32)
    _expect(beta, "beta", (B, T, H), f32)
    _expect(S0, "S0", (B, H, dv, dk), f32, required=False)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=bf, device=q.device)
    _expect(o, "o", (B, T, H, dv), bf)
    if S_out is None and return_state:
        S_out = torch.empty((B, H, dv, dk), dtype=f32, device=q.device)
    _expect(S_out, "S_out", (B, H, dv, dk), f32, required=False)
    a = PermArgs()
    a.B, a.T, a.H, a.dk, a.dv = B, T, H, dk, dv
    a.q, a.k, a.v, a.src, a.beta, a.w = map(_ptr, (q, k, v, src, beta, w))
    a.S0, a.o, a.S_out = _ptr(S0), _ptr(o), _ptr(S_out)
    _check(call_perm_fwd(a, _stream(stream)))
    return o, S_out


# ------------------------------------------------------------ channelwise operators
GDR_SCAN_BLOCK = 32       # tokens between two saved states (include/gdr_scan.h)
GDR_CKPT8_GROUP = 128     # values that share one exponent (include/gdr_ckpt8.h)
GDR_SSM_BLOCK = 32        # tokens between two saved states (include/gdr_ssm.h)


class ScanArgs(ctypes.Structure):
    """Mirror of ``gdr_scan_args`` (include/gdr_scan.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("C", _i32), ("io_dtype", _i32),
        ("x", _vp), ("alpha", _vp), ("decay_x", _vp), ("decay_a", _vp), ("gate_x", _vp),
        ("normalise", _i32), ("reserved", _i32), ("h0", _vp), ("y", _vp), ("h_out", _vp),
        ("ckpt", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class ScanBwdArgs(ctypes.Structure):
    """Mirror of ``gdr_scan_bwd_args`` (include/gdr_scan.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("C", _i32), ("io_dtype", _i32),
        ("x", _vp), ("x_exp", _vp), ("alpha", _vp), ("decay_x", _vp), ("decay_a", _vp),
        ("gate_x", _vp), ("normalise", _i32), ("reserved", _i32), ("h0", _vp), ("ckpt", _vp),
        ("grad_y", _vp), ("grad_h", _vp), ("grad_x", _vp), ("grad_alpha", _vp),
        ("grad_decay_x", _vp), ("grad_decay_a", _vp), ("grad_gate_x", _vp), ("grad_h0", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class ScanStepArgs(ctypes.Structure):
    """Mirror of ``gdr_scan_step_args`` (include/gdr_scan.h)."""
    _fields_ = [
        ("N", _i32), ("C", _i32), ("io_dtype", _i32), ("normalise", _i32),
        ("x", _vp), ("alpha", _vp), ("decay_x", _vp), ("decay_a", _vp), ("gate_x", _vp),
        ("h", _vp), ("h_out", _vp), ("y", _vp),
    ]


class NormArgs(ctypes.Structure):
    """Mirror of ``gdr_norm_args`` (include/gdr_norm.h)."""
    _fields_ = [
        ("R", ctypes.c_int64), ("D", _i32), ("io_dtype", _i32), ("eps", ctypes.c_float),
        ("reserved", _i32), ("x", _vp), ("weight", _vp), ("bias", _vp), ("y", _vp),
        ("mean", _vp), ("rstd", _vp), ("x_code", _vp), ("x_exp", _vp),
    ]


class NormBwdArgs(ctypes.Structure):
    """Mirror of ``gdr_norm_bwd_args`` (include/gdr_norm.h)."""
    _fields_ = [
        ("R", ctypes.c_int64), ("D", _i32), ("io_dtype", _i32),
        ("x", _vp), ("x_exp", _vp), ("mean", _vp), ("rstd", _vp), ("weight", _vp),
        ("grad_y", _vp), ("grad_x", _vp), ("grad_weight", _vp), ("grad_bias", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class Ckpt8PackArgs(ctypes.Structure):
    """Mirror of ``gdr_ckpt8_pack_args`` (include/gdr_ckpt8.h)."""
    _fields_ = [("R", ctypes.c_int64), ("D", _i32), ("io_dtype", _i32),
                ("x", _vp), ("code", _vp), ("exp", _vp)]


class Ckpt8UnpackArgs(ctypes.Structure):
    """Mirror of ``gdr_ckpt8_unpack_args`` (include/gdr_ckpt8.h)."""
    _fields_ = [("R", ctypes.c_int64), ("D", _i32), ("io_dtype", _i32),
                ("code", _vp), ("exp", _vp), ("x", _vp)]


class ConvArgs(ctypes.Structure):
    """Mirror of ``gdr_conv_args`` (include/gdr_conv.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("C", _i32), ("K", _i32), ("io_dtype", _i32), ("silu", _i32),
        ("x", _vp), ("weight", _vp), ("bias", _vp), ("state", _vp), ("lens", _vp), ("y", _vp), ("state_out", _vp),
    ]


class ConvBwdArgs(ctypes.Structure):
    """Mirror of ``gdr_conv_bwd_args`` (include/gdr_conv.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("C", _i32), ("K", _i32), ("io_dtype", _i32), ("silu", _i32),
        ("x", _vp), ("weight", _vp), ("bias", _vp), ("state", _vp), ("lens", _vp), ("grad_y", _vp),
        ("grad_state_out", _vp), ("grad_x", _vp), ("grad_weight", _vp), ("grad_bias", _vp), ("grad_state", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class ConvStepArgs(ctypes.Structure):
    """Mirror of ``gdr_conv_step_args`` (include/gdr_conv.h)."""
    _fields_ = [
        ("N", _i32), ("C", _i32), ("K", _i32), ("io_dtype", _i32), ("silu", _i32), ("reserved", _i32),
        ("x", _vp), ("weight", _vp), ("bias", _vp), ("state", _vp), ("state_out", _vp), ("y", _vp),
    ]


class SsmArgs(ctypes.Structure):
    """Mirror of ``gdr_ssm_args`` (include/gdr_ssm.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("C", _i32), ("N", _i32), ("G", _i32), ("io_dtype", _i32), ("softplus", _i32),
        ("reserved", _i32), ("x", _vp), ("dt", _vp), ("A", _vp), ("Bv", _vp), ("Cv", _vp), ("D", _vp), ("z", _vp),
        ("dt_bias", _vp), ("h0", _vp), ("lens", _vp), ("y", _vp), ("h_out", _vp), ("ckpt", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class SsmBwdArgs(ctypes.Structure):
    """Mirror of ``gdr_ssm_bwd_args`` (include/gdr_ssm.h)."""
    _fields_ = [
        ("B", _i32), ("T", _i32), ("C", _i32), ("N", _i32), ("G", _i32), ("io_dtype", _i32), ("softplus", _i32),
        ("reserved", _i32), ("x", _vp), ("dt", _vp), ("A", _vp), ("Bv", _vp), ("Cv", _vp), ("D", _vp), ("z", _vp),
        ("dt_bias", _vp), ("h0", _vp), ("ckpt", _vp), ("lens", _vp), ("grad_y", _vp), ("grad_h", _vp),
        ("grad_x", _vp), ("grad_dt", _vp), ("grad_A", _vp), ("grad_Bv", _vp), ("grad_Cv", _vp), ("grad_D", _vp),
        ("grad_z", _vp), ("grad_dt_bias", _vp), ("grad_h0", _vp), ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class SsmStepArgs(ctypes.Structure):
    """Mirror of ``gdr_ssm_step_args`` (include/gdr_ssm.h)."""
    _fields_ = [
        ("R", _i32), ("C", _i32), ("N", _i32), ("G", _i32), ("io_dtype", _i32), ("softplus", _i32),
        ("x", _vp), ("dt", _vp), ("A", _vp), ("Bv", _vp), ("Cv", _vp), ("D", _vp), ("z", _vp), ("dt_bias", _vp),
        ("h", _vp), ("h_out", _vp), ("y", _vp),
    ]


class GnormArgs(ctypes.Structure):
    """Mirror of ``gdr_gnorm_args`` (include/gdr_gnorm.h)."""
    _fields_ = [
        ("R", ctypes.c_int64), ("C", _i32), ("G", _i32), ("io_dtype", _i32), ("center", _i32), ("silu", _i32),
        ("eps", ctypes.c_float), ("x", _vp), ("z", _vp), ("weight", _vp), ("bias", _vp), ("y", _vp),
        ("mean", _vp), ("rstd", _vp),
    ]


class GnormBwdArgs(ctypes.Structure):
    """Mirror of ``gdr_gnorm_bwd_args`` (include/gdr_gnorm.h)."""
    _fields_ = [
        ("R", ctypes.c_int64), ("C", _i32), ("G", _i32), ("io_dtype", _i32), ("silu", _i32),
        ("x", _vp), ("z", _vp), ("mean", _vp), ("rstd", _vp), ("weight", _vp), ("bias", _vp), ("grad_y", _vp),
        ("grad_x", _vp), ("grad_z", _vp), ("grad_weight", _vp), ("grad_bias", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


_CHANNELWISE = {"gdr_scan_fwd": ScanArgs, "gdr_scan_bwd": ScanBwdArgs,
                "gdr_scan_step": ScanStepArgs, "gdr_norm_fwd": NormArgs,
                "gdr_norm_bwd": NormBwdArgs, "gdr_ckpt8_pack": Ckpt8PackArgs,
                "gdr_ckpt8_unpack": Ckpt8UnpackArgs,
                "gdr_conv_fwd": ConvArgs, "gdr_conv_bwd": ConvBwdArgs, "gdr_conv_step": ConvStepArgs,
                "gdr_ssm_fwd": SsmArgs, "gdr_ssm_bwd": SsmBwdArgs, "gdr_ssm_step": SsmStepArgs,
                "gdr_gnorm_fwd": GnormArgs, "gdr_gnorm_bwd": GnormBwdArgs}
_CHANNELWISE_WS = {"gdr_scan_fwd_workspace": ScanArgs, "gdr_scan_bwd_workspace": ScanBwdArgs,
                   "gdr_norm_bwd_workspace": NormBwdArgs, "gdr_conv_bwd_workspace": ConvBwdArgs,
                   "gdr_ssm_fwd_workspace": SsmArgs, "gdr_ssm_bwd_workspace": SsmBwdArgs,
                   "gdr_gnorm_bwd_workspace": GnormBwdArgs}


def call_channelwise(name: str, args, stream=None) -> int:
    """Raw call of a channelwise entry point (the keys of ``_CHANNELWISE``:
    ``gdr_scan_fwd``, ``gdr_norm_fwd``, ``gdr_conv_fwd``, ``gdr_ssm_fwd``, ...) with its
    filled struct; returns the status code."""
    s = stream if isinstance(stream, ctypes.c_void_p) else (
        ctypes.c_void_p(0) if stream is None else _stream(stream))
    return getattr(load_library(), name)(ctypes.byref(args), s)


def _in(t, name, shape, dtype, dev):
    """Device pointer of one argument after checking its shape, dtype, contiguity
    and device (``_expect`` and ``_ptr`` in one, cheap enough for single-token calls)."""
    if t is None or t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        _expect(t, name, shape, dtype)
    if t.device != dev:
        if not t.is_cuda:
            raise ValueError("gdr: tensors must live on the GPU")
        raise ValueError(f"gdr: {name} is on {t.device}, expected {dev}")
    return t.data_ptr()


def _opt(t, name, shape, dtype, dev):
    return None if t is None else _in(t, name, shape, dtype, dev)


def _elsewhere(dev, stream) -> bool:
    """Whether a call on ``dev`` has to leave the current device or stream."""
    import torch
    return stream is not None or dev.type != "cuda" or dev.index != torch._C._cuda_getDevice()


def _there(dev, stream):
    """Context of a call that has to: ``stream``, which must belong to ``dev``, or the
    current stream of ``dev``.  Outputs and workspaces are allocated inside, so that the
    allocator ties them to the stream that uses them."""
    import torch
    if dev.type != "cuda":
        raise ValueError("gdr: tensors must live on the GPU")
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"gdr: stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _launch(entry, args, dev):
    import torch
    _check(entry(ctypes.byref(args), torch._C._cuda_getCurrentRawStream(dev.index)))


def _workspace(need, workspace, dev):
    """(pointer, bytes) of a workspace of ``need`` bytes, and the tensor that owns it."""
    import torch
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif (workspace.dtype != torch.uint8 or workspace.numel() < need or workspace.device != dev
          or not workspace.is_contiguous()):
        raise ValueError(f"gdr: workspace must be a contiguous uint8 tensor of at least {need} bytes on {dev}")
    return workspace.data_ptr(), workspace.numel(), workspace


def _x8(x, lead, D, dev):
    """Pointers of an 8-bit checkpoint (codes, exponents) of shape [*lead, D]."""
    import torch
    code, exp = x
    return (_in(code, "x[0]", (*lead, D), torch.float8_e4m3fn, dev),
            _in(exp, "x[1]", (*lead, -(-D // GDR_CKPT8_GROUP)), torch.uint8, dev))


def _scan_fwd(x, alpha, decay_x, decay_a, gate_x, normalise, h0, y, h_out, ckpt, return_state, return_ckpt,
              workspace, stream):
    import torch
    if x.dim() != 3:
        raise ValueError("gdr: x must be [B,T,C]")
    shape, io, f32, dev = x.shape, x.dtype, torch.float32, x.device
    B, T, C = shape
    code_io = _io(x)
    xp = _in(x, "x", shape, io, dev)
    ap = dp = sp = gp = None
    if alpha is not None:
        ap = _in(alpha, "alpha", shape, f32, dev)
    else:
        dp = _in(decay_x, "decay_x", shape, io, dev)
        sp = _in(decay_a, "decay_a", (C,), f32, dev)
        gp = _opt(gate_x, "gate_x", shape, io, dev)
    hp = _opt(h0, "h0", (B, C), f32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return _scan_fwd(x, alpha, decay_x, decay_a, gate_x, normalise, h0, y, h_out, ckpt, return_state, return_ckpt,
                             workspace, None)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    op = cp = None
    if h_out is not None:
        op = _in(h_out, "h_out", (B, C), f32, dev)
    elif return_state:
        h_out = torch.empty((B, C), dtype=f32, device=dev)
        op = h_out.data_ptr()
    cshape = (B, -(-T // GDR_SCAN_BLOCK), C)
    if ckpt is not None:
        cp = _in(ckpt, "ckpt", cshape, f32, dev)
    elif return_ckpt:
        ckpt = torch.empty(cshape, dtype=f32, device=dev)
        cp = ckpt.data_ptr()
    lib = load_library()
    a = ScanArgs(B, T, C, code_io, xp, ap, dp, sp, gp, int(alpha is None and bool(normalise)), 0, hp, yp, op, cp)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_scan_fwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_scan_fwd, a, dev)
    return y, h_out, ckpt


def gdr_scan_fwd(x, alpha, *, h0=None, y=None, h_out=None, ckpt=None, return_state=True,
                 return_ckpt=False, workspace=None, stream=None):
    """Channelwise linear recurrence h_t = alpha_t h_{t-1} + x_t, y_t = h_t (see
    ``gdr_scan_fwd`` in include/gdr_scan.h).

    x [B,T,C] bf16 or fp32; alpha fp32 [B,T,C] in [0, 1] (0 starts anew); h0 fp32
    [B,C] or None (zero).  Returns (y [B,T,C] like x, h_out fp32 [B,C], ckpt) --
    h_out None unless ``return_state`` or given (it may be h0), ckpt fp32
    [B,ceil(T/32),C] (the states before each 32 tokens, for the backward) None
    unless ``return_ckpt`` or given.  The workspace (``gdr_scan_fwd_workspace``
    bytes) is allocated here unless a large enough uint8 tensor is passed, which
    serves one call at a time.
    """
    if alpha is None:
        raise ValueError("gdr: alpha is required")
    return _scan_fwd(x, alpha, None, None, None, False, h0, y, h_out, ckpt, return_state, return_ckpt, workspace,
                     stream)


def gdr_scan_fwd_gated(x, decay_x, decay_a, *, gate_x=None, normalise=True, h0=None, y=None,
                       h_out=None, ckpt=None, return_state=True, return_ckpt=False, workspace=None,
                       stream=None):
    """The recurrence with its gates computed in the kernel (include/gdr_scan.h):
    u = decay_a softplus(decay_x), h_t = exp(-u_t) h_{t-1} + b_t x_t with
    b = sigmoid(gate_x) (1 without gate_x), times sqrt(1 - exp(-2 u)) with ``normalise``.

    x, decay_x, gate_x [B,T,C], all bf16 or all fp32; decay_a fp32 [C], >= 0; the
    rest and the results as ``gdr_scan_fwd``.
    """
    if decay_x is None or decay_a is None:
        raise ValueError("gdr: decay_x and decay_a are required")
    return _scan_fwd(x, None, decay_x, decay_a, gate_x, normalise, h0, y, h_out, ckpt, return_state, return_ckpt,
                     workspace, stream)


def _scan_bwd(x, alpha, decay_x, decay_a, gate_x, normalise, grad_y, h0, grad_h, ckpt, need_grad_h0, workspace,
              stream):
    import torch
    if grad_y.dim() != 3:
        raise ValueError("gdr: grad_y must be [B,T,C]")
    shape, io, f32, dev = grad_y.shape, grad_y.dtype, torch.float32, grad_y.device
    B, T, C = shape
    code_io = _io(grad_y)
    xp, ep = _x8(x, (B, T), C, dev) if isinstance(x, tuple) else (_in(x, "x", shape, io, dev), None)
    ap = dp = sp = gp = None
    if alpha is not None:
        ap = _in(alpha, "alpha", shape, f32, dev)
    else:
        dp = _in(decay_x, "decay_x", shape, io, dev)
        sp = _in(decay_a, "decay_a", (C,), f32, dev)
        gp = _opt(gate_x, "gate_x", shape, io, dev)
    if ckpt is not None and h0 is not None:
        raise ValueError("gdr: pass either ckpt or h0, not both (ckpt holds the start state)")
    hp = _opt(h0, "h0", (B, C), f32, dev)
    cp = _opt(ckpt, "ckpt", (B, -(-T // GDR_SCAN_BLOCK), C), f32, dev)
    gyp = _in(grad_y, "grad_y", shape, io, dev)
    ghp = _opt(grad_h, "grad_h", (B, C), f32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return _scan_bwd(x, alpha, decay_x, decay_a, gate_x, normalise, grad_y, h0, grad_h, ckpt, need_grad_h0,
                             workspace, None)
    g = {"x": torch.empty_like(grad_y)}
    gal = gdx = gda = ggx = gh0 = None
    if alpha is not None:
        g["alpha"] = torch.empty_like(alpha)
        gal = g["alpha"].data_ptr()
    else:
        g["decay_x"] = torch.empty_like(decay_x)
        g["decay_a"] = torch.empty_like(decay_a)
        gdx, gda = g["decay_x"].data_ptr(), g["decay_a"].data_ptr()
        if gate_x is not None:
            g["gate_x"] = torch.empty_like(gate_x)
            ggx = g["gate_x"].data_ptr()
    if need_grad_h0:
        g["h0"] = torch.empty((B, C), dtype=f32, device=dev)
        gh0 = g["h0"].data_ptr()
    lib = load_library()
    a = ScanBwdArgs(B, T, C, code_io, xp, ep, ap, dp, sp, gp, int(alpha is None and bool(normalise)), 0, hp, cp, gyp,
                    ghp, g["x"].data_ptr(), gal, gdx, gda, ggx, gh0)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_scan_bwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_scan_bwd, a, dev)
    return g


def gdr_scan_bwd(x, alpha, grad_y, *, h0=None, grad_h=None, ckpt=None, need_grad_h0=True,
                 workspace=None, stream=None):
    """Gradients of ``gdr_scan_fwd`` (``gdr_scan_bwd`` in include/gdr_scan.h).

    x, alpha and h0 as the forward's; grad_y [B,T,C] like x, grad_h fp32 [B,C] or
    None.  ``ckpt`` (the forward's, in place of h0) saves the second run of the
    recurrence.  x may be an 8-bit checkpoint, the tuple ``gdr_ckpt8_pack``
    returned.  Returns a dict: x (like grad_y), alpha (fp32) and, when
    ``need_grad_h0``, h0 (fp32).  The workspace (``gdr_scan_bwd_workspace``
    bytes) is allocated here unless a large enough uint8 tensor is passed, which
    serves one call at a time.
    """
    if alpha is None:
        raise ValueError("gdr: alpha is required")
    return _scan_bwd(x, alpha, None, None, None, False, grad_y, h0, grad_h, ckpt, need_grad_h0, workspace, stream)


def gdr_scan_bwd_gated(x, decay_x, decay_a, grad_y, *, gate_x=None, normalise=True, h0=None, grad_h=None,
                       ckpt=None, need_grad_h0=True, workspace=None, stream=None):
    """Gradients of ``gdr_scan_fwd_gated``; arguments as there and as
    ``gdr_scan_bwd``.  Returns a dict: x, decay_x and (with gate_x) gate_x like
    grad_y, decay_a fp32 [C] and, when ``need_grad_h0``, h0 fp32 [B,C]."""
    if decay_x is None or decay_a is None:
        raise ValueError("gdr: decay_x and decay_a are required")
    return _scan_bwd(x, None, decay_x, decay_a, gate_x, normalise, grad_y, h0, grad_h, ckpt, need_grad_h0, workspace,
                     stream)


def _scan_step(h, x, alpha, decay_x, decay_a, gate_x, normalise, h_out, y, stream):
    import torch
    if x.dim() != 2:
        raise ValueError("gdr: x must be [N,C]")
    shape, io, f32, dev = x.shape, x.dtype, torch.float32, x.device
    N, C = shape
    code_io = _io(x)
    if h_out is None:
        h_out = h
    hp = _in(h, "h", shape, f32, dev)
    xp = _in(x, "x", shape, io, dev)
    ho = hp if h_out is h else _in(h_out, "h_out", shape, f32, dev)
    if alpha is not None:
        gates = (_in(alpha, "alpha", shape, f32, dev), None, None, None)
    else:
        gates = (None, _in(decay_x, "decay_x", shape, io, dev), _in(decay_a, "decay_a", (C,), f32, dev),
                 _opt(gate_x, "gate_x", shape, io, dev))
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return _scan_step(h, x, alpha, decay_x, decay_a, gate_x, normalise, h_out, y, None)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    a = ScanStepArgs(N, C, code_io, int(bool(normalise)), xp, *gates, hp, ho, yp)
    _launch(load_library().gdr_scan_step, a, dev)
    return y


def gdr_scan_step(h, x, alpha, *, h_out=None, y=None, stream=None):
    """One token of ``gdr_scan_fwd`` on N states (``gdr_scan_step`` in
    include/gdr_scan.h).  h [N,C] fp32, overwritten unless ``h_out`` is given;
    x [N,C] bf16 or fp32, alpha fp32 [N,C].  Returns y [N,C] like x."""
    if alpha is None:
        raise ValueError("gdr: alpha is required")
    return _scan_step(h, x, alpha, None, None, None, False, h_out, y, stream)


def gdr_scan_step_gated(h, x, decay_x, decay_a, *, gate_x=None, normalise=True, h_out=None, y=None,
                        stream=None):
    """One token of ``gdr_scan_fwd_gated`` on N states: x, decay_x, gate_x [N,C],
    decay_a fp32 [C], the rest as ``gdr_scan_step``."""
    if decay_x is None or decay_a is None:
        raise ValueError("gdr: decay_x and decay_a are required")
    return _scan_step(h, x, None, decay_x, decay_a, gate_x, normalise, h_out, y, stream)


def gdr_norm_fwd(x, weight=None, bias=None, *, eps=1e-5, y=None, return_stats=True, return_ckpt8=False,
                 stream=None):
    """Layer norm over the last dimension (see ``gdr_norm_fwd`` in include/gdr_norm.h).

    x [...,D] bf16 or fp32; weight, bias fp32 [D] or None.  Returns (y like x,
    mean, rstd, ckpt8): the statistics fp32 [...] (None without ``return_stats``),
    and with ``return_ckpt8`` the 8-bit copy of x for the backward (the tuple of
    ``gdr_ckpt8_pack``), else None.
    """
    import torch
    if x.dim() < 1:
        raise ValueError("gdr: x must be [...,D]")
    shape, io, f32, dev = x.shape, x.dtype, torch.float32, x.device
    lead, D = shape[:-1], shape[-1]
    R, code_io = math.prod(lead), _io(x)
    xp = _in(x, "x", shape, io, dev)
    wp = _opt(weight, "weight", (D,), f32, dev)
    bp = _opt(bias, "bias", (D,), f32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_norm_fwd(x, weight, bias, eps=eps, y=y, return_stats=return_stats, return_ckpt8=return_ckpt8)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    mean = rstd = mp = rp = None
    if return_stats:
        mean = torch.empty(lead, dtype=f32, device=dev)
        rstd = torch.empty(lead, dtype=f32, device=dev)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    code, kept = (None, None), None
    if return_ckpt8:
        kept = (torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev),
                torch.empty((*lead, -(-D // GDR_CKPT8_GROUP)), dtype=torch.uint8, device=dev))
        code = kept[0].data_ptr(), kept[1].data_ptr()
    a = NormArgs(R, D, code_io, eps, 0, xp, wp, bp, yp, mp, rp, *code)
    _launch(load_library().gdr_norm_fwd, a, dev)
    return y, mean, rstd, kept


def gdr_norm_bwd(grad_y, x, mean, rstd, weight=None, *, need_grad_weight=True, need_grad_bias=True,
                 workspace=None, stream=None):
    """Gradients of ``gdr_norm_fwd`` (``gdr_norm_bwd`` in include/gdr_norm.h).

    grad_y [...,D]; x like it, or the forward's ckpt8 tuple; mean, rstd and weight
    as the forward's.  Returns a dict: x like grad_y, and weight and bias fp32 [D]
    unless not needed.  The workspace (``gdr_norm_bwd_workspace`` bytes) is
    allocated here unless a large enough uint8 tensor is passed.
    """
    import torch
    if grad_y.dim() < 1:
        raise ValueError("gdr: grad_y must be [...,D]")
    shape, io, f32, dev = grad_y.shape, grad_y.dtype, torch.float32, grad_y.device
    lead, D = shape[:-1], shape[-1]
    R, code_io = math.prod(lead), _io(grad_y)
    xp, ep = _x8(x, lead, D, dev) if isinstance(x, tuple) else (_in(x, "x", shape, io, dev), None)
    mp, rp = _in(mean, "mean", lead, f32, dev), _in(rstd, "rstd", lead, f32, dev)
    wp = _opt(weight, "weight", (D,), f32, dev)
    gyp = _in(grad_y, "grad_y", shape, io, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_norm_bwd(grad_y, x, mean, rstd, weight, need_grad_weight=need_grad_weight,
                                need_grad_bias=need_grad_bias, workspace=workspace)
    g = {"x": torch.empty_like(grad_y)}
    gwp = gbp = None
    if need_grad_weight:
        g["weight"] = torch.empty((D,), dtype=f32, device=dev)
        gwp = g["weight"].data_ptr()
    if need_grad_bias:
        g["bias"] = torch.empty((D,), dtype=f32, device=dev)
        gbp = g["bias"].data_ptr()
    lib = load_library()
    a = NormBwdArgs(R, D, code_io, xp, ep, mp, rp, wp, gyp, g["x"].data_ptr(), gwp, gbp)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_norm_bwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_norm_bwd, a, dev)
    return g


def gdr_ckpt8_pack(x, *, stream=None):
    """8-bit checkpoint of an activation (``gdr_ckpt8_pack`` in include/gdr_ckpt8.h):
    x [...,D] bf16 or fp32 -> (codes float8_e4m3fn [...,D], exponents uint8
    [...,ceil(D/128)]), each code standing for code * 2^(exponent - 127)."""
    import torch
    if x.dim() < 1:
        raise ValueError("gdr: x must be [...,D]")
    shape, dev = x.shape, x.device
    lead, D = shape[:-1], shape[-1]
    code_io = _io(x)
    xp = _in(x, "x", shape, x.dtype, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_ckpt8_pack(x)
    code = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    exp = torch.empty((*lead, -(-D // GDR_CKPT8_GROUP)), dtype=torch.uint8, device=dev)
    a = Ckpt8PackArgs(math.prod(lead), D, code_io, xp, code.data_ptr(), exp.data_ptr())
    _launch(load_library().gdr_ckpt8_pack, a, dev)
    return code, exp


def gdr_ckpt8_unpack(code, exp, *, dtype=None, x=None, stream=None):
    """The values of an 8-bit checkpoint (``gdr_ckpt8_unpack`` in include/gdr_ckpt8.h),
    in ``dtype`` (bf16 by default, or fp32), written to ``x`` when given."""
    import torch
    if code.dim() < 1:
        raise ValueError("gdr: the codes must be [...,D]")
    shape, dev = code.shape, code.device
    lead, D = shape[:-1], shape[-1]
    if dtype is None:
        dtype = torch.bfloat16 if x is None else x.dtype
    cp = _in(code, "code", shape, torch.float8_e4m3fn, dev)
    ep = _in(exp, "exp", (*lead, -(-D // GDR_CKPT8_GROUP)), torch.uint8, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_ckpt8_unpack(code, exp, dtype=dtype, x=x)
    if x is None:
        x = torch.empty(shape, dtype=dtype, device=dev)
        xp = x.data_ptr()
    else:
        xp = _in(x, "x", shape, dtype, dev)
    a = Ckpt8UnpackArgs(math.prod(lead), D, _io(x), cp, ep, xp)
    _launch(load_library().gdr_ckpt8_unpack, a, dev)
    return x


# ------------------------------------------------------------ short causal convolution
def _taps(weight, bias, C, dev):
    """(K, pointers of weight and bias) of a convolution over C channels."""
    import torch
    if weight is None or weight.dim() != 2:
        raise ValueError("gdr: weight must be [C,K]")
    K = weight.shape[1]
    return K, _in(weight, "weight", (C, K), torch.float32, dev), _opt(bias, "bias", (C,), torch.float32, dev)


def _edge(K):
    """Rows of a convolution's state (the C layer refuses the taps that have none)."""
    return max(K - 1, 0)


def gdr_conv_fwd(x, weight, bias=None, *, state=None, lens=None, silu=True, y=None, state_out=None,
                 return_state=True, stream=None):
    """Short causal convolution of every channel over its last K tokens, with silu unless
    ``silu`` is false (see ``gdr_conv_fwd`` in include/gdr_conv.h).

    x [B,T,C] bf16 or fp32; weight fp32 [C,K], 2 <= K <= 8, its last column for the token
    itself; bias fp32 [C] or None; state [B,K-1,C] like x, the tokens before the first, or
    None (zeros); lens int32 [B], the tokens of each row of a padded batch, or None (T).
    Returns (y like x, state_out [B,K-1,C]: the last K-1 inputs of each row, None unless
    ``return_state`` or given; it may be state)."""
    import torch
    if x.dim() != 3:
        raise ValueError("gdr: x must be [B,T,C]")
    shape, io, dev = x.shape, x.dtype, x.device
    B, T, C = shape
    code_io = _io(x)
    xp = _in(x, "x", shape, io, dev)
    K, wp, bp = _taps(weight, bias, C, dev)
    edge = (B, _edge(K), C)
    sp = _opt(state, "state", edge, io, dev)
    lp = _opt(lens, "lens", (B,), torch.int32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_conv_fwd(x, weight, bias, state=state, lens=lens, silu=silu, y=y, state_out=state_out,
                                return_state=return_state)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    op = None
    if state_out is not None:
        op = _in(state_out, "state_out", edge, io, dev)
    elif return_state:
        state_out = torch.empty(edge, dtype=io, device=dev)
        op = state_out.data_ptr()
    a = ConvArgs(B, T, C, K, code_io, int(bool(silu)), xp, wp, bp, sp, lp, yp, op)
    _launch(load_library().gdr_conv_fwd, a, dev)
    return y, state_out


def gdr_conv_bwd(grad_y, x, weight, bias=None, *, state=None, lens=None, silu=True, grad_state=None,
                 need_grad_state=True, workspace=None, stream=None):
    """Gradients of ``gdr_conv_fwd`` (``gdr_conv_bwd`` in include/gdr_conv.h); x to silu as
    the forward's, grad_y like x, grad_state like state: the gradient of state_out, or None.

    Returns a dict: x like grad_y, weight fp32 [C,K], bias fp32 [C] (with bias) and, when
    ``need_grad_state``, state like grad_y [B,K-1,C].  The workspace
    (``gdr_conv_bwd_workspace`` bytes) is allocated here unless a large enough uint8 tensor
    is passed, which serves one call at a time."""
    import torch
    if grad_y.dim() != 3:
        raise ValueError("gdr: grad_y must be [B,T,C]")
    shape, io, f32, dev = grad_y.shape, grad_y.dtype, torch.float32, grad_y.device
    B, T, C = shape
    code_io = _io(grad_y)
    gp = _in(grad_y, "grad_y", shape, io, dev)
    xp = _in(x, "x", shape, io, dev)
    K, wp, bp = _taps(weight, bias, C, dev)
    edge = (B, _edge(K), C)
    sp = _opt(state, "state", edge, io, dev)
    lp = _opt(lens, "lens", (B,), torch.int32, dev)
    gsp = _opt(grad_state, "grad_state", edge, io, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_conv_bwd(grad_y, x, weight, bias, state=state, lens=lens, silu=silu, grad_state=grad_state,
                                need_grad_state=need_grad_state, workspace=workspace)
    g = {"x": torch.empty_like(grad_y), "weight": torch.empty((C, K), dtype=f32, device=dev)}
    gbp = gop = None
    if bias is not None:
        g["bias"] = torch.empty((C,), dtype=f32, device=dev)
        gbp = g["bias"].data_ptr()
    if need_grad_state:
        g["state"] = torch.empty(edge, dtype=io, device=dev)
        gop = g["state"].data_ptr()
    lib = load_library()
    a = ConvBwdArgs(B, T, C, K, code_io, int(bool(silu)), xp, wp, bp, sp, lp, gp, gsp, g["x"].data_ptr(),
                    g["weight"].data_ptr(), gbp, gop)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_conv_bwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_conv_bwd, a, dev)
    return g


def gdr_conv_step(state, x, weight, bias=None, *, silu=True, state_out=None, y=None, stream=None):
    """One token of ``gdr_conv_fwd`` on N states (``gdr_conv_step`` in include/gdr_conv.h).
    state [N,K-1,C] like x [N,C], overwritten unless ``state_out`` is given; weight fp32
    [C,K], bias fp32 [C] or None.  Returns y like x."""
    import torch
    if x.dim() != 2:
        raise ValueError("gdr: x must be [N,C]")
    shape, io, dev = x.shape, x.dtype, x.device
    N, C = shape
    code_io = _io(x)
    xp = _in(x, "x", shape, io, dev)
    K, wp, bp = _taps(weight, bias, C, dev)
    edge = (N, _edge(K), C)
    sp = _in(state, "state", edge, io, dev)
    op = sp if state_out is None or state_out is state else _in(state_out, "state_out", edge, io, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_conv_step(state, x, weight, bias, silu=silu, state_out=state_out, y=y)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    a = ConvStepArgs(N, C, K, code_io, int(bool(silu)), 0, xp, wp, bp, sp, op, yp)
    _launch(load_library().gdr_conv_step, a, dev)
    return y


# ------------------------------------------------------------ selective state space scan
def _ssm_inputs(ref, lead, x, dt, A, B, C, D, z, dt_bias):
    """(N, G, pointers in the structs' order) of a scan whose rows are ``lead`` and whose
    activations are like ``ref``."""
    import torch
    io, f32, dev = ref.dtype, torch.float32, ref.device
    chans = ref.shape[-1]
    if A is None or A.dim() != 2:
        raise ValueError("gdr: A must be [C,N]")
    if B is None or B.dim() != len(lead) + 2:
        raise ValueError("gdr: B must be [%s,G,N]" % ("B,T" if len(lead) == 2 else "R"))
    N, G = A.shape[1], B.shape[-2]
    vec = (*lead, G, N)
    return N, G, (_in(x, "x", ref.shape, io, dev), _in(dt, "dt", ref.shape, io, dev), _in(A, "A", (chans, N), f32, dev),
                  _in(B, "B", vec, io, dev), _in(C, "C", vec, io, dev), _opt(D, "D", (chans,), f32, dev),
                  _opt(z, "z", ref.shape, io, dev), _opt(dt_bias, "dt_bias", (chans,), f32, dev))


def gdr_ssm_fwd(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, h0=None, lens=None, y=None,
                h_out=None, ckpt=None, return_state=True, return_ckpt=False, workspace=None, stream=None):
    """Selective state space scan (see ``gdr_ssm_fwd`` in include/gdr_ssm.h): with
    d = softplus(dt + dt_bias), h_t = exp(d_t A) h_{t-1} + d_t x_t B_t and
    y_t = (C_t . h_t + D x_t) silu(z_t).

    x, dt, z [B,T,C] and B, C [B,T,G,N], all bf16 or all fp32 (each group's vectors serve
    C / G neighbouring channels); A fp32 [C,N], N <= 64; D, dt_bias fp32 [C] or None; h0 fp32
    [B,C,N] or None (zero); lens int32 [B], the tokens of each row of a padded batch, or
    None (T).  Without ``softplus`` d is dt + dt_bias.  Returns (y like x, h_out fp32
    [B,C,N], ckpt) -- h_out None unless ``return_state`` or given (it may be h0), ckpt fp32
    [B,ceil(T/32),N,C] (the states before each 32 tokens, for the backward) None unless
    ``return_ckpt`` or given.  The workspace (``gdr_ssm_fwd_workspace`` bytes) is allocated
    here unless a large enough uint8 tensor is passed, which serves one call at a time."""
    import torch
    if x.dim() != 3:
        raise ValueError("gdr: x must be [B,T,C]")
    shape, io, f32, dev = x.shape, x.dtype, torch.float32, x.device
    nb, T, chans = shape
    code_io = _io(x)
    N, G, ins = _ssm_inputs(x, (nb, T), x, dt, A, B, C, D, z, dt_bias)
    hshape = (nb, chans, N)
    hp = _opt(h0, "h0", hshape, f32, dev)
    lp = _opt(lens, "lens", (nb,), torch.int32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_ssm_fwd(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus, h0=h0, lens=lens, y=y,
                               h_out=h_out, ckpt=ckpt, return_state=return_state, return_ckpt=return_ckpt,
                               workspace=workspace)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    op = cp = None
    if h_out is not None:
        op = _in(h_out, "h_out", hshape, f32, dev)
    elif return_state:
        h_out = torch.empty(hshape, dtype=f32, device=dev)
        op = h_out.data_ptr()
    cshape = (nb, -(-T // GDR_SSM_BLOCK), N, chans)
    if ckpt is not None:
        cp = _in(ckpt, "ckpt", cshape, f32, dev)
    elif return_ckpt:
        ckpt = torch.empty(cshape, dtype=f32, device=dev)
        cp = ckpt.data_ptr()
    lib = load_library()
    a = SsmArgs(nb, T, chans, N, G, code_io, int(bool(softplus)), 0, *ins, hp, lp, yp, op, cp)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_ssm_fwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_ssm_fwd, a, dev)
    return y, h_out, ckpt


def gdr_ssm_bwd(grad_y, x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, h0=None, lens=None,
                grad_h=None, ckpt=None, need_grad_h0=True, workspace=None, stream=None):
    """Gradients of ``gdr_ssm_fwd`` (``gdr_ssm_bwd`` in include/gdr_ssm.h); x to lens as the
    forward's, grad_y like x, grad_h fp32 [B,C,N] (of h_out) or None.  ``ckpt`` (the
    forward's, in place of h0) saves the second run of the recurrence.

    Returns a dict: x, dt, B, C and (with z) z like the inputs; A fp32 [C,N] and (with them)
    D, dt_bias fp32 [C]; when ``need_grad_h0``, h0 fp32 [B,C,N].  The workspace
    (``gdr_ssm_bwd_workspace`` bytes) is allocated here unless a large enough uint8 tensor
    is passed, which serves one call at a time."""
    import torch
    if grad_y.dim() != 3:
        raise ValueError("gdr: grad_y must be [B,T,C]")
    shape, io, f32, dev = grad_y.shape, grad_y.dtype, torch.float32, grad_y.device
    nb, T, chans = shape
    code_io = _io(grad_y)
    N, G, ins = _ssm_inputs(grad_y, (nb, T), x, dt, A, B, C, D, z, dt_bias)
    hshape = (nb, chans, N)
    if ckpt is not None and h0 is not None:
        raise ValueError("gdr: pass either ckpt or h0, not both (ckpt holds the start state)")
    hp = _opt(h0, "h0", hshape, f32, dev)
    cp = _opt(ckpt, "ckpt", (nb, -(-T // GDR_SSM_BLOCK), N, chans), f32, dev)
    lp = _opt(lens, "lens", (nb,), torch.int32, dev)
    gp = _in(grad_y, "grad_y", shape, io, dev)
    ghp = _opt(grad_h, "grad_h", hshape, f32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_ssm_bwd(grad_y, x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus, h0=h0, lens=lens,
                               grad_h=grad_h, ckpt=ckpt, need_grad_h0=need_grad_h0, workspace=workspace)
    g = {"x": torch.empty_like(grad_y), "dt": torch.empty_like(grad_y), "A": torch.empty_like(A),
         "B": torch.empty_like(B), "C": torch.empty_like(B)}
    gD = gz = gb = gh0 = None
    if D is not None:
        g["D"] = torch.empty_like(D)
        gD = g["D"].data_ptr()
    if z is not None:
        g["z"] = torch.empty_like(z)
        gz = g["z"].data_ptr()
    if dt_bias is not None:
        g["dt_bias"] = torch.empty_like(dt_bias)
        gb = g["dt_bias"].data_ptr()
    if need_grad_h0:
        g["h0"] = torch.empty(hshape, dtype=f32, device=dev)
        gh0 = g["h0"].data_ptr()
    lib = load_library()
    a = SsmBwdArgs(nb, T, chans, N, G, code_io, int(bool(softplus)), 0, *ins, hp, cp, lp, gp, ghp,
                   g["x"].data_ptr(), g["dt"].data_ptr(), g["A"].data_ptr(), g["B"].data_ptr(), g["C"].data_ptr(),
                   gD, gz, gb, gh0)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_ssm_bwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_ssm_bwd, a, dev)
    return g


def gdr_ssm_step(h, x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, h_out=None, y=None, stream=None):
    """One token of ``gdr_ssm_fwd`` on R states (``gdr_ssm_step`` in include/gdr_ssm.h).
    h fp32 [R,C,N], overwritten unless ``h_out`` is given; x, dt, z [R,C], B, C [R,G,N], the
    rest as there.  Returns y like x."""
    import torch
    if x.dim() != 2:
        raise ValueError("gdr: x must be [R,C]")
    shape, io, f32, dev = x.shape, x.dtype, torch.float32, x.device
    R, chans = shape
    code_io = _io(x)
    N, G, ins = _ssm_inputs(x, (R,), x, dt, A, B, C, D, z, dt_bias)
    hp = _in(h, "h", (R, chans, N), f32, dev)
    op = hp if h_out is None or h_out is h else _in(h_out, "h_out", (R, chans, N), f32, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_ssm_step(h, x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus, h_out=h_out, y=y)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    a = SsmStepArgs(R, chans, N, G, code_io, int(bool(softplus)), *ins, hp, op, yp)
    _launch(load_library().gdr_ssm_step, a, dev)
    return y


# ------------------------------------------------------------ gated group norm
def gdr_gnorm_fwd(x, groups, weight=None, bias=None, *, z=None, silu=False, center=True, eps=1e-5, y=None,
                  return_stats=True, stream=None):
    """Group norm over ``groups`` equal runs of the last dimension, with an activation or a
    gate (see ``gdr_gnorm_fwd`` in include/gdr_gnorm.h): u = xh weight + bias, and
    y = u act(z) with z, else act(u), where act is silu or nothing.  Without ``center`` no
    mean is taken off.

    x, z [...,C] bf16 or fp32; weight, bias fp32 [C] or None.  Returns (y like x, mean,
    rstd): the statistics fp32 [...,groups] (None without ``return_stats``, mean None
    without ``center``)."""
    import torch
    if x.dim() < 1:
        raise ValueError("gdr: x must be [...,C]")
    shape, io, f32, dev = x.shape, x.dtype, torch.float32, x.device
    lead, chans, G = shape[:-1], shape[-1], operator.index(groups)
    R, code_io = math.prod(lead), _io(x)
    xp = _in(x, "x", shape, io, dev)
    zp = _opt(z, "z", shape, io, dev)
    wp = _opt(weight, "weight", (chans,), f32, dev)
    bp = _opt(bias, "bias", (chans,), f32, dev)
    if G < 1 or chans % G:
        raise ValueError(f"gdr: {chans} channels do not fall into {groups} groups")
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_gnorm_fwd(x, groups, weight, bias, z=z, silu=silu, center=center, eps=eps, y=y,
                                 return_stats=return_stats)
    if y is None:
        y = torch.empty_like(x)
        yp = y.data_ptr()
    else:
        yp = _in(y, "y", shape, io, dev)
    mean = rstd = mp = rp = None
    if return_stats:
        rstd = torch.empty((*lead, G), dtype=f32, device=dev)
        rp = rstd.data_ptr()
        if center:
            mean = torch.empty((*lead, G), dtype=f32, device=dev)
            mp = mean.data_ptr()
    a = GnormArgs(R, chans, G, code_io, int(bool(center)), int(bool(silu)), eps, xp, zp, wp, bp, yp, mp, rp)
    _launch(load_library().gdr_gnorm_fwd, a, dev)
    return y, mean, rstd


def gdr_gnorm_bwd(grad_y, x, mean, rstd, groups, weight=None, bias=None, *, z=None, silu=False,
                  need_grad_weight=True, need_grad_bias=True, workspace=None, stream=None):
    """Gradients of ``gdr_gnorm_fwd`` (``gdr_gnorm_bwd`` in include/gdr_gnorm.h); grad_y like
    x, the statistics as the forward returned them (mean None: it took none off), the rest
    as the forward's.  Returns a dict: x and (with z) z like grad_y, and weight and bias
    fp32 [C] unless not needed.  The workspace (``gdr_gnorm_bwd_workspace`` bytes) is
    allocated here unless a large enough uint8 tensor is passed."""
    import torch
    if grad_y.dim() < 1:
        raise ValueError("gdr: grad_y must be [...,C]")
    shape, io, f32, dev = grad_y.shape, grad_y.dtype, torch.float32, grad_y.device
    lead, chans, G = shape[:-1], shape[-1], operator.index(groups)
    R, code_io = math.prod(lead), _io(grad_y)
    if G < 1 or chans % G:
        raise ValueError(f"gdr: {chans} channels do not fall into {groups} groups")
    gp = _in(grad_y, "grad_y", shape, io, dev)
    xp = _in(x, "x", shape, io, dev)
    mp, rp = _opt(mean, "mean", (*lead, G), f32, dev), _in(rstd, "rstd", (*lead, G), f32, dev)
    wp = _opt(weight, "weight", (chans,), f32, dev)
    bp = _opt(bias, "bias", (chans,), f32, dev)
    zp = _opt(z, "z", shape, io, dev)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gdr_gnorm_bwd(grad_y, x, mean, rstd, groups, weight, bias, z=z, silu=silu,
                                 need_grad_weight=need_grad_weight, need_grad_bias=need_grad_bias, workspace=workspace)
    g = {"x": torch.empty_like(grad_y)}
    gzp = gwp = gbp = None
    if z is not None:
        g["z"] = torch.empty_like(grad_y)
        gzp = g["z"].data_ptr()
    if need_grad_weight:
        g["weight"] = torch.empty((chans,), dtype=f32, device=dev)
        gwp = g["weight"].data_ptr()
    if need_grad_bias:
        g["bias"] = torch.empty((chans,), dtype=f32, device=dev)
        gbp = g["bias"].data_ptr()
    lib = load_library()
    a = GnormBwdArgs(R, chans, G, code_io, int(bool(silu)), xp, zp, mp, rp, wp, bp, gp, g["x"].data_ptr(), gzp, gwp, gbp)
    a.workspace, a.workspace_bytes, keep = _workspace(
        lib.gdr_gnorm_bwd_workspace(ctypes.byref(a)), workspace, dev)
    _launch(lib.gdr_gnorm_bwd, a, dev)
    return g
