"""GPTQ layer-wise weight quantization on NVIDIA B200 (sm_100a).

The hot path runs in libgptq_b200.so (C ABI in include/gptq.h and include/fp8.h); this package is
its binding (`_lib` and `_fp8`, same names as the C entry points) plus small allocation
helpers (`layer`, `fp8`) and the data-parallel driver over torch.distributed (`sharded`).
Importing it without the built library raises: there is no CPU fallback. The 8-bit floating point calls
come with a binding of their own; where that cannot be loaded, using them raises.
"""
from ._lib import (EXPORTED, GPTQ_BF16, GPTQ_F32, GPTQ_ORDER_DESC_ACT, GPTQ_ORDER_GIVEN,  # noqa: F401
                   GPTQ_ORDER_NATURAL, GPTQError, LIB_PATH, gptq_hessian_accumulate,
                   gptq_dequant_gemm, gptq_dequant_gemv, gptq_gemm_f32, gptq_pack, gptq_params, gptq_prepare_hinv, gptq_quantize_layer, gptq_quantize_pack_layer,
                   gptq_quantize_layer_noalloc, GPTQ_NOALLOC_SCRATCH_BYTES,
                   gptq_status_string, gptq_workspace_size, make_params, rtn_quantize, status_string)
from .layer import QuantizedLayer, check_status, hessian, prepare, quantize_layer, rtn  # noqa: F401
from . import sharded  # noqa: F401  (token-sharded H, one all-reduce, row-sharded sweep)

try:
    from ._fp8 import (EXPORTED_FP8, GPTQ_F16, fp8_add_rmsnorm, fp8_gated_gemm, fp8_gemm,  # noqa: F401
                       fp8_quantize)
    from . import fp8  # noqa: F401  (layers held in e4m3 with block scales)
except ImportError as e:  # the other calls need the library alone: only the use of these raises
    _fp8_error = str(e)

    def __getattr__(name):
        if name in ("EXPORTED_FP8", "GPTQ_F16", "fp8", "fp8_add_rmsnorm", "fp8_gated_gemm", "fp8_gemm",
                    "fp8_quantize"):
            raise ImportError(_fp8_error)
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
