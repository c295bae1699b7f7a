"""The C ABI of the 8-bit floating point operators: what include/fp8.h declares is exported and
bound, and bad arguments are rejected on the host before anything is launched (no GPU)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
V, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
FAKE = 0x1000   # aligned, never dereferenced: every call below returns before a launch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    lib = ctypes.CDLL(__graft_entry__._build_module().build())
    lib.fp8_quantize.argtypes = [V, I32, I64, I64, I64, I32, V, I64, V, I64, V]
    lib.fp8_add_rmsnorm.argtypes = [V, I64, V, I64, I32, V, I32, F32, I64, I64, V, I64, V, I64, V,
                                    I64, V]
    lib.fp8_gemm.argtypes = [V, I64, V, I64] * 2 + [I64] * 3 + [V, I32, I64, V, V]
    lib.fp8_gated_gemm.argtypes = [V, I64, V, I64] * 3 + [I64] * 3 + [V, I64, V, I64, V, V]
    return lib


def caller(fn, ok):
    def call(**kw):
        assert set(kw) <= set(ok), kw
        return fn(*{**ok, **kw}.values())
    return call


def test_header_binding_and_exports_agree(lib):
    import post_weight_quantization_18_b200 as G
    src = open(os.path.join(ROOT, "include", "fp8.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(re.findall(r"^int (\w+)\s*\(", src, flags=re.M))
    assert names == sorted(G.EXPORTED_FP8) and len(names) == 4
    for name in names:
        assert hasattr(lib, name) and callable(getattr(G, name)), name


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_is_plain_c99(tmp_path):
    src = tmp_path / "c.c"
    src.write_text('#include "fp8.h"\nint main(void) { return fp8_quantize(0, GPTQ_F16, 1, 0, 0, 1, '
                   '0, 1, 0, 1, 0) == GPTQ_ERR_INVALID_ARG ? 0 : 1; }\n')
    import post_weight_quantization_18_b200 as G
    libdir = os.path.dirname(G.LIB_PATH)
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "c"),
                        "-L", libdir, "-l:" + os.path.basename(G.LIB_PATH),
                        "-Wl,-rpath," + libdir], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(tmp_path / "c")], timeout=60).returncode == 0


def test_quantize_refusals(lib):
    call = caller(lib.fp8_quantize, dict(X=FAKE, t=0, ldx=300, m=8, k=300, rows=1, Q=FAKE, ldq=304,
                                         s=FAKE, lds=3, stream=None))
    assert call(X=None) == 1 and call(Q=None) == 1 and call(s=None) == 1
    assert call(m=-1) == 1 and call(k=0) == 1 and call(m=(1 << 30) + 1) == 1
    assert call(ldx=299) == 1 and call(ldq=299) == 1 and call(lds=2) == 1
    assert call(rows=64) == 1 and call(rows=0) == 1
    assert call(t=3) == 2 and call(t=-1) == 2
    assert call(X=FAKE + 1) == 1 and call(t=1, X=FAKE + 2) == 1 and call(s=FAKE + 2) == 1
    assert call(m=0) == 0 and call(m=0, X=None, Q=None, s=None) == 0


def test_norm_refusals(lib):
    call = caller(lib.fp8_add_rmsnorm,
                  dict(X=FAKE, ldx=256, R=FAKE * 2, ldr=256, t=0, g=FAKE, gt=0, eps=1e-5, m=4, k=256,
                       H=FAKE * 3, ldh=256, Q=FAKE * 4, ldq=256, s=FAKE * 5, lds=2, stream=None))
    assert call(X=None) == 1 and call(g=None) == 1 and call(Q=None) == 1 and call(s=None) == 1
    assert call(ldx=255) == 1 and call(ldr=255) == 1 and call(ldh=255) == 1 and call(ldq=255) == 1
    assert call(lds=1) == 1 and call(k=0) == 1 and call(m=-1) == 1
    assert call(eps=-1e-6) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(t=5) == 2 and call(gt=2) == 2            # gamma: the rows' type or fp32
    assert call(H=FAKE, ldh=512) == 1                    # in place with another pitch
    assert call(H=FAKE * 2, ldh=512) == 1
    assert call(R=FAKE * 2 + 1) == 1 and call(H=FAKE * 3 + 1) == 1 and call(gt=1, g=FAKE + 2) == 1
    assert call(m=0) == 0 and call(m=0, X=None, R=None, H=None, Q=None, s=None) == 0


def test_gemm_refusals(lib):
    call = caller(lib.fp8_gemm,
                  dict(X=FAKE, ldx=256, sx=FAKE, ldsx=2, W=FAKE, ldw=256, sw=FAKE, ldsw=2, m=4, n=300,
                       k=256, Y=FAKE, t=0, ldy=300, st=None, stream=None))
    for name in ("X", "sx", "W", "sw", "Y"):
        assert call(**{name: None}) == 1, name
    for name, v in (("ldx", 255), ("ldsx", 1), ("ldw", 255), ("ldsw", 1), ("ldy", 299)):
        assert call(**{name: v}) == 1, name
    assert call(m=-1) == 1 and call(n=0) == 1 and call(k=0) == 1 and call(n=(1 << 30) + 1) == 1
    assert call(t=4) == 2
    assert call(sx=FAKE + 1) == 1 and call(Y=FAKE + 1) == 1 and call(t=1, Y=FAKE + 2) == 1
    assert call(st=FAKE + 2) == 1
    assert call(m=0) == 0 and call(m=0, X=None, Y=None) == 0


def test_gated_refusals(lib):
    call = caller(lib.fp8_gated_gemm,
                  dict(X=FAKE, ldx=256, sx=FAKE, ldsx=2, Wg=FAKE, ldg=256, sg=FAKE, ldsg=2, Wu=FAKE,
                       ldu=256, su=FAKE, ldsu=2, m=4, n=300, k=256, Q=FAKE, ldq=300, s=FAKE, lds=3,
                       st=None, stream=None))
    for name in ("X", "sx", "Wg", "sg", "Wu", "su", "Q", "s"):
        assert call(**{name: None}) == 1, name
    for name, v in (("ldx", 255), ("ldsx", 1), ("ldg", 255), ("ldsg", 1), ("ldu", 255), ("ldsu", 1),
                    ("ldq", 299), ("lds", 2)):
        assert call(**{name: v}) == 1, name
    assert call(m=-1) == 1 and call(n=0) == 1 and call(k=0) == 1
    assert call(s=FAKE + 2) == 1 and call(su=FAKE + 1) == 1
    assert call(m=0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """The Python checks come before any CUDA call."""
    import post_weight_quantization_18_b200 as G
    q = torch.zeros((4, 256), dtype=torch.uint8)
    s = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        G.fp8_quantize(torch.zeros((4, 256)), q, s)
    with pytest.raises(ValueError, match="block_rows"):
        G.fp8_quantize(torch.zeros((4, 256)), q, s, 64)
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        G.fp8_quantize(torch.zeros((4, 256), dtype=torch.float64), q, s)
    with pytest.raises(ValueError, match="2 dims"):
        G.fp8_gemm(q[0], s, q, s, torch.zeros((4, 4)))
    with pytest.raises(ValueError, match="CUDA"):
        G.fp8_gemm(q, s, q, s, torch.zeros((4, 4)))
    x = G.fp8.FP8Matrix(q.view(torch.float8_e4m3fn), s, 1)
    with pytest.raises(ValueError, match="128 x 128"):
        G.fp8.linear(x, x)
