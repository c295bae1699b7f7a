"""Binding of the 8-bit floating point operators (include/fp8.h) — argument marshalling only.

As in `_lib`, every function has the name of the C entry point it calls, takes torch CUDA tensors
(outputs included), checks them on the host (ValueError), runs on the current stream of their device
and raises GPTQError on a non-OK return. e4m3 matrices are torch.float8_e4m3fn or torch.uint8
tensors. The functions are those of csrc/fp8_binding.cpp; there is no fallback: without the built
extension importing this module raises.
"""
from __future__ import annotations

import os

from . import _lib

try:
    from . import _fp8_binding
except ImportError as e:
    raise ImportError(
        f"{os.path.join(os.path.dirname(_lib.LIB_PATH), '_fp8_binding.so')} cannot be loaded ({e}): "
        "build it with `python post_weight_quantization_18_b200/build.py` (there is no CPU fallback)"
    ) from e

GPTQ_F16 = 2

EXPORTED_FP8 = ("fp8_quantize", "fp8_add_rmsnorm", "fp8_gemm", "fp8_gated_gemm")

_fp8_binding.set_error(_lib.GPTQError)
fp8_quantize = _fp8_binding.fp8_quantize
fp8_add_rmsnorm = _fp8_binding.fp8_add_rmsnorm
fp8_gemm = _fp8_binding.fp8_gemm
fp8_gated_gemm = _fp8_binding.fp8_gated_gemm
