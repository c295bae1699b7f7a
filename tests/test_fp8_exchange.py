"""The room that the products of few rows count for the sums of a cluster holds them all."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_room_for_the_sums_of_a_cluster(tmp_path):
    """Every place that a CTA of a cluster writes its sums to lies inside the area counted for them."""
    exe = tmp_path / "fp8_exchange_check"
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-I",
                        os.path.join(ROOT, "post_weight_quantization_18_b200", "csrc"),
                        os.path.join(ROOT, "tests", "c", "fp8_exchange_check.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe), "16", "32", "64"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "0", r.stdout
