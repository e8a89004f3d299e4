"""How a warp of the Muon products takes accumulators in turn when the products
stop for good: rr_ring.h compiled for the host against a model of the barriers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_tile_counts_after_a_wait_that_ran_out(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = tmp_path / "ring_check"
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "allgather_rr_allreduce_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "native", "ring_check.cpp"), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout + res.stderr
