"""The loads of 4-bit weights stay inside their operands: the kernels' offsets,
compiled for the host and walked over odd widths, lengths and first blocks."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "mixture_experts_routed_route_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_loads_of_4_bit_weights(tmp_path):
    exe = str(tmp_path / "walk")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "q4_addr_walk.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("ok")
