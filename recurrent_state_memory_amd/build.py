"""Build libgdr.so (HIP for gfx950) in-tree with hipcc.

    python -m recurrent_state_memory_amd.build [--jobs N]

Every HIP source is compiled for gfx950 only.  Packed-fp32 VALU instructions
are disabled for all device code (``-packed-fp32-ops``); hipcc's host pass
warns that it does not know that feature, which is harmless.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libgdr.so")

SOURCES = ["gdr_api.cpp", "gdr_fwd.hip", "gdr_fwd_pipe.hip", "gdr_step.hip", "gdr_bwd.hip", "gdr_gate_bwd.hip", "gdr_noalloc.hip",
           "raven_api.cpp", "raven_fwd.hip", "perm_api.cpp", "perm_fwd.hip",
           "scan_api.cpp", "scan_fwd.hip", "scan_bwd.hip", "norm_api.cpp", "norm.hip", "ckpt8.hip",
           "conv_api.cpp", "conv.hip", "ssm_api.cpp", "ssm_fwd.hip", "ssm_bwd.hip", "gnorm_api.cpp", "gnorm.hip"]

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wno-unused-result",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CFLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(ln for ln in r.stderr.splitlines() if noise not in ln)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        print(err, file=sys.stderr)
    return obj


def build(jobs: int = 4, verbose: bool = True) -> str:
    """Compile every source and link ``libgdr.so`` next to this file."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=min(8, os.cpu_count() or 4))
    a = ap.parse_args(argv)
    build(a.jobs)


if __name__ == "__main__":
    main()
