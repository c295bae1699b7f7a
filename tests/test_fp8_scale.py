"""The scale's division by 448, as the kernels do it, is the correctly rounded one: every mantissa,
at ordinary exponents, the largest, and the smallest whose quotient is a normal number."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_division_by_448_on_every_mantissa(tmp_path):
    exe = tmp_path / "fp8_scale_check"
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-mfma", "-ffp-contract=off", "-Wall", "-Werror",
                        "-Wno-unknown-pragmas", "-I",
                        os.path.join(ROOT, "post_weight_quantization_18_b200", "csrc"),
                        os.path.join(ROOT, "tests", "c", "fp8_scale_check.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe), "0", "-20", "9", "127", "-117"], capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "0", r.stdout
