"""Binding of the 8-bit floating point operators (include/fp8.h) — argument marshalling only.

As in `_lib`, every function has the name of the C entry point it calls, takes torch CUDA tensors
(outputs included), checks them on the host (ValueError), runs on the current stream of their device
and raises GPTQError on a non-OK return. e4m3 matrices are torch.float8_e4m3fn or torch.uint8
tensors. The functions are those of csrc/fp8_binding.cpp; there is no fallback: without the built
extension importing this module raises.
"""
from __future__ import annotations

import os
import re
import sys

import torch

from . import _lib


def _load():
    """The extension module, compiled for the torch and Python at hand: it reads objects by their layout."""
    try:
        from . import _fp8_binding
    except ImportError as e:
        why = e
    else:
        version = re.match(r"[0-9.]*[0-9]", torch.__version__).group()
        here = f"torch {version}, Python {sys.version_info.major}.{sys.version_info.minor}"
        built_for = getattr(_fp8_binding, "built_for", "an earlier version")
        if here == built_for:
            return _fp8_binding
        why = f"it was built for {built_for}, this is {here}"
    raise ImportError(
        f"{os.path.join(os.path.dirname(_lib.LIB_PATH), '_fp8_binding.so')} cannot be loaded ({why}): "
        "build it with `python post_weight_quantization_18_b200/build.py` (there is no CPU fallback)")


_fp8_binding = _load()

GPTQ_F16 = 2

EXPORTED_FP8 = ("fp8_quantize", "fp8_add_rmsnorm", "fp8_gemm", "fp8_gated_gemm")

_fp8_binding.set_error(_lib.GPTQError)
fp8_quantize = _fp8_binding.fp8_quantize
fp8_add_rmsnorm = _fp8_binding.fp8_add_rmsnorm
fp8_gemm = _fp8_binding.fp8_gemm
fp8_gated_gemm = _fp8_binding.fp8_gated_gemm
