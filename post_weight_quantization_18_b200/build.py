"""Build libgptq_b200.so in-tree with nvcc for sm_100a.

    python post_weight_quantization_18_b200/build.py          # rebuild if sources changed
    python post_weight_quantization_18_b200/build.py --force

(Run it as a script, not as `python -m`: importing the package loads the library.)

Each .cu under csrc/ is compiled to an object (in parallel) and the objects are linked into one
shared library next to this file. The CUDA runtime is linked statically; the driver API is
reached through cudaGetDriverEntryPoint, so libcuda is not a link-time dependency.
csrc/fp8_binding.cpp is compiled against the Python and torch headers into _fp8_binding.so, the
extension module that calls the library's 8-bit floating point operators.
"""
from __future__ import annotations

import fcntl
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgptq_b200.so")
BINDING = os.path.join(HERE, "_fp8_binding.so")
BINDING_SRC = os.path.join(CSRC, "fp8_binding.cpp")
BINDING_FOR = os.path.join(OBJDIR, "_fp8_binding.for")   # the torch and Python it was compiled for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def binding_abi() -> str:
    """What the binding's machine code depends on beside its source: torch's C++ layout and Python's."""
    return f"torch {importlib.metadata.version('torch')} {sysconfig.get_config_var('SOABI')}\n"


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        if f.read() != binding_abi():
            return False
    t = os.path.getmtime(BINDING)
    return all(os.path.getmtime(p) <= t
               for p in [BINDING_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))])


def build_binding() -> None:
    """_fp8_binding.so from csrc/fp8_binding.cpp (the library has to be there: it is linked)."""
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(binding_abi())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date() and binding_up_to_date():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    with open(os.path.join(OBJDIR, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)   # until closed: processes that build at once take turns
        build_library(force, verbose)
        if force or not binding_up_to_date():
            build_binding()
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
