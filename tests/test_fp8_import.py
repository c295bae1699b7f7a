"""The e4m3 operators' binding is an extension module of its own. Without it, or with one built for another
torch, the calls of the integer formats import as before, and the e4m3 ones say what is missing."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "post_weight_quantization_18_b200"
PKG = os.path.join(ROOT, NAME)

USE = f"""
import {NAME} as G
assert callable(G.gptq_dequant_gemv) and callable(G.quantize_layer) and callable(G.rtn) and G.sharded
for use in (lambda: G.fp8_quantize, lambda: G.fp8_gemm, lambda: G.fp8, lambda: G.EXPORTED_FP8,
            lambda: __import__("{NAME}.fp8"), lambda: exec("from {NAME} import fp8_gemm")):
    try:
        use()
        print("no error")
    except ImportError as e:
        assert "_fp8_binding.so" in str(e) and "build" in str(e), e
try:
    G.fp9
except AttributeError:
    print("ok")
"""


def copy_of_package(tmp_path, binding=None):
    dst = tmp_path / NAME
    dst.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py"):
            shutil.copy(os.path.join(PKG, name), dst / name)
    os.symlink(os.path.join(PKG, "libgptq_b200.so"), dst / "libgptq_b200.so")
    if binding is not None:
        os.symlink(binding, dst / "_fp8_binding.so")
    return dst


def run(tmp_path, code):
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                          timeout=300, env={**os.environ, "PYTHONPATH": str(tmp_path)})


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    return __graft_entry__._build_module().build()


def test_integer_formats_without_the_binding(tmp_path):
    copy_of_package(tmp_path)
    r = run(tmp_path, USE)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_everything_with_the_binding(tmp_path):
    copy_of_package(tmp_path, os.path.join(PKG, "_fp8_binding.so"))
    r = run(tmp_path, f"import {NAME} as G; print(callable(G.fp8_gemm), G.fp8.__name__)")
    assert r.returncode == 0 and r.stdout.strip() == f"True {NAME}.fp8", r.stdout + r.stderr


def test_binding_of_another_torch_is_refused(tmp_path):
    """It reads tensors by the layout it was compiled against. Without a torch of another version at hand, the
    version that this one reports is changed."""
    copy_of_package(tmp_path, os.path.join(PKG, "_fp8_binding.so"))
    r = run(tmp_path, "import torch; torch.__version__ = '1.13.1+cu117'\n" + USE)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_binding_is_rebuilt_for_another_torch_or_python(built, monkeypatch):
    import importlib.metadata
    import sysconfig

    import __graft_entry__
    build = __graft_entry__._build_module()
    assert build.binding_up_to_date()
    with monkeypatch.context() as mp:
        version = importlib.metadata.version
        mp.setattr(importlib.metadata, "version", lambda n: "1.13.1" if n == "torch" else version(n))
        assert not build.binding_up_to_date()
    with monkeypatch.context() as mp:
        get = sysconfig.get_config_var
        mp.setattr(sysconfig, "get_config_var", lambda n: "cpython-38" if n == "SOABI" else get(n))
        assert not build.binding_up_to_date()
    assert build.binding_up_to_date()


def test_binding_that_does_not_say_what_it_was_built_for(tmp_path):
    """One from before it did, left by an update of the sources without a build."""
    dst = copy_of_package(tmp_path)
    (dst / "_fp8_binding.py").write_text("def set_error(e): pass\n")
    r = run(tmp_path, USE)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
