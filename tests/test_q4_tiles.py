"""Launches and tiles of products of many rows on 4-bit weights: the kernel's own
arithmetic, compiled for the host and walked over up to the largest sizes."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "mixture_experts_routed_route_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_launches_and_tiles(tmp_path):
    exe = str(tmp_path / "walk")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "q4_tiles_walk.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("ok")
