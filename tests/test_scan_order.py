"""The order in which the channelwise recurrence's workgroups take its tiles, on the CPU
(tests/scan_order_harness.cpp): whole and ragged teams of chains, one tile and many."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_tile_once_and_after_those_it_waits_for(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "order"
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "recurrent_state_memory_amd", "csrc"),
                    os.path.join(ROOT, "tests", "scan_order_harness.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and "SCAN_ORDER_OK" in out.stdout, out.stdout + out.stderr
