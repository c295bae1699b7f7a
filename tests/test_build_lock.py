"""Two processes that build at once (two test runs, a build beside an import) do not write one another's
files: with stand-ins for the compilers that refuse to write what another one is writing."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

TOOL = """#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = -o ] && out=$2; shift; done
mkdir "$out.busy" || exit 1
echo x >> "$(dirname "$0")/calls"
sleep 0.3
echo built > "$out"
rmdir "$out.busy"
"""


@pytest.mark.skipif(not os.path.exists("/bin/sh"), reason="needs a shell")
def test_builds_take_turns(tmp_path):
    pkg, bin_ = tmp_path / "pkg", tmp_path / "bin"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    bin_.mkdir()
    shutil.copy(os.path.join(ROOT, "post_weight_quantization_18_b200", "build.py"), pkg / "build.py")
    for name in ("a.cu", "b.cu", "fp8_binding.cpp"):
        (pkg / "csrc" / name).write_text("")
    for name in ("nvcc", "g++"):
        (bin_ / name).write_text(TOOL)
        (bin_ / name).chmod(0o755)
    env = {**os.environ, "NVCC": str(bin_ / "nvcc"), "PATH": f"{bin_}:{os.environ['PATH']}"}
    ps = [subprocess.Popen([sys.executable, str(pkg / "build.py")], env=env, stdout=subprocess.PIPE,
                           stderr=subprocess.STDOUT, text=True) for _ in range(3)]
    outs = [p.communicate(timeout=300)[0] for p in ps]
    assert [p.returncode for p in ps] == [0, 0, 0], outs
    assert (pkg / "libgptq_b200.so").read_text() == (pkg / "_fp8_binding.so").read_text() == "built\n"
    # two objects, the library, the binding: once, as the second process found them up to date
    assert (bin_ / "calls").read_text().count("x") == 4
