"""The two-at-a-time square roots and quotients of the 8-bit AdamW step round
as the device's own: every mantissa of square roots and reciprocals, random
quotients (tests/native/rounding_check.cu, built and run here)."""
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_roots_and_quotients_are_correctly_rounded(tmp_path):
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    from allgather_rr_allreduce_gb300 import build
    exe = tmp_path / "rounding_check"
    subprocess.run([build._nvcc()] + build.ARCH + ["-O3", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(ROOT, "tests", "native", "rounding_check.cu"), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "square roots off: 0, quotients off: 0, reciprocals off: 0" in res.stdout
