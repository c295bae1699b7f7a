"""ctypes binding of the 8-bit floating point operators (include/fp8.h) — argument marshalling only.

As in `_lib`, every function has the name of the C entry point it calls, takes torch CUDA tensors
(outputs included), checks them on the host, runs on the current stream of their device and raises
GPTQError on a non-OK return. e4m3 matrices are torch.float8_e4m3fn or torch.uint8 tensors.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import GPTQ_BF16, GPTQ_F32, _check, _lib

GPTQ_F16 = 2

EXPORTED_FP8 = ("fp8_quantize", "fp8_add_rmsnorm", "fp8_gemm", "fp8_gated_gemm")

_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_lib.fp8_quantize.argtypes = [_P, _I32, _I64, _I64, _I64, _I32, _P, _I64, _P, _I64, _P]
_lib.fp8_add_rmsnorm.argtypes = [_P, _I64, _P, _I64, _I32, _P, _I32, _F32, _I64, _I64, _P, _I64,
                                 _P, _I64, _P, _I64, _P]
_lib.fp8_gemm.argtypes = [_P, _I64, _P, _I64] * 2 + [_I64] * 3 + [_P, _I32, _I64, _P, _P]
_lib.fp8_gated_gemm.argtypes = [_P, _I64, _P, _I64] * 3 + [_I64] * 3 + [_P, _I64, _P, _I64, _P, _P]
for _name in EXPORTED_FP8:
    getattr(_lib, _name).restype = _I32

_DTYPES = {torch.bfloat16: GPTQ_BF16, torch.float32: GPTQ_F32, torch.float16: GPTQ_F16}
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def _matrix(t: torch.Tensor, name: str, rows: int, cols: int, pitch: int = 1) -> int:
    """The leading dimension of t, a [rows, cols] CUDA tensor with unit stride along its rows. One
    row alone has no pitch: it counts as the next multiple of `pitch`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its last dim")
    if rows <= 1:
        return -(-cols // pitch) * pitch
    return ld


def _e4m3(t: torch.Tensor, name: str, rows: int, cols: int) -> int:
    if t.dtype not in _E4M3:
        raise ValueError(f"{name} must be float8_e4m3fn or uint8, got {t.dtype}")
    return _matrix(t, name, rows, cols, 16)


def _scales(t: torch.Tensor, name: str, rows: int, cols: int) -> int:
    if t.dtype is not torch.float32:
        raise ValueError(f"{name} must be torch.float32, got {t.dtype}")
    return _matrix(t, name, rows, cols)


def _float_code(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _shape2(t: torch.Tensor, name: str) -> tuple[int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor of 2 dims")
    return t.shape[0], t.shape[1]


def _status_ptr(t: torch.Tensor | None, dev: torch.device):
    if t is None:
        return None
    if not t.is_cuda or t.device != dev or t.dtype is not torch.int32 or t.numel() < 2 \
            or not t.is_contiguous():
        raise ValueError("dev_status must be a contiguous int32 CUDA tensor of 2 entries on the "
                         "operands' device")
    return t.data_ptr()


def _call(fn, where: str, dev: torch.device, others, *args) -> None:
    """fn(*args, stream) with the tensors' device current (they must share one)."""
    for t in others:
        if t.device != dev:
            raise ValueError(f"{where}: tensors are on different devices ({dev} and {t.device})")
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    if rc:
        _check(rc, where)


def fp8_quantize(X: torch.Tensor, Q: torch.Tensor, scales: torch.Tensor, block_rows: int = 1
                 ) -> None:
    """Q, scales = X [m, k] as e4m3 with one fp32 scale per 1 x 128 (activations) or 128 x 128
    (weights, block_rows=128) block."""
    m, k = _shape2(X, "X")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    code = _float_code(X, "X")
    ldx = _matrix(X, "X", m, k, 8)
    ldq = _e4m3(Q, "Q", m, k)
    lds = _scales(scales, "scales", -(-m // block_rows), -(-k // 128))
    _call(_lib.fp8_quantize, "fp8_quantize", X.device, (Q, scales), X.data_ptr(), code, ldx, m, k,
          block_rows, Q.data_ptr(), ldq, scales.data_ptr(), lds)


def fp8_add_rmsnorm(X: torch.Tensor, R: torch.Tensor | None, gamma: torch.Tensor, eps: float,
                    H: torch.Tensor | None, Q: torch.Tensor, scales: torch.Tensor) -> None:
    """h = X + R; H = h (may be X or R itself); Q, scales = h / sqrt(mean(h^2) + eps) * gamma as
    e4m3 with one scale per row and 128 columns. R and H may be None."""
    m, k = _shape2(X, "X")
    code = _float_code(X, "X")
    gcode = _float_code(gamma, "gamma")
    ldx = _matrix(X, "X", m, k, 8)
    if not gamma.is_cuda or gamma.dim() != 1 or gamma.shape[0] != k or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous CUDA tensor of k entries")
    others = [gamma, Q, scales]
    r_ptr = h_ptr = None
    ldr = ldh = 0
    if R is not None:
        if R.dtype is not X.dtype:
            raise ValueError("R must have X's dtype")
        ldr = _matrix(R, "R", m, k, 8)
        r_ptr = R.data_ptr()
        others.append(R)
    if H is not None:
        if H.dtype is not X.dtype:
            raise ValueError("H must have X's dtype")
        ldh = _matrix(H, "H", m, k, 8)
        h_ptr = H.data_ptr()
        others.append(H)
    ldq = _e4m3(Q, "Q", m, k)
    lds = _scales(scales, "scales", m, -(-k // 128))
    _call(_lib.fp8_add_rmsnorm, "fp8_add_rmsnorm", X.device, others, X.data_ptr(), ldx, r_ptr, ldr,
          code, gamma.data_ptr(), gcode, float(eps), m, k, h_ptr, ldh, Q.data_ptr(), ldq,
          scales.data_ptr(), lds)


def fp8_gemm(X: torch.Tensor, sx: torch.Tensor, W: torch.Tensor, sw: torch.Tensor,
             Y: torch.Tensor, dev_status: torch.Tensor | None = None) -> None:
    """Y [m, n] (bf16, fp16 or fp32) = X W^T of X [m, k] (blocks of 1 x 128, scales sx) and W [n, k]
    (blocks of 128 x 128, scales sw)."""
    m, k = _shape2(X, "X")
    n = _shape2(W, "W")[0]
    g = -(-k // 128)
    ldx, ldsx = _e4m3(X, "X", m, k), _scales(sx, "sx", m, g)
    ldw, ldsw = _e4m3(W, "W", n, k), _scales(sw, "sw", -(-n // 128), g)
    code = _float_code(Y, "Y")
    ldy = _matrix(Y, "Y", m, n, 8)
    _call(_lib.fp8_gemm, "fp8_gemm", X.device, (sx, W, sw, Y), X.data_ptr(), ldx, sx.data_ptr(),
          ldsx, W.data_ptr(), ldw, sw.data_ptr(), ldsw, m, n, k, Y.data_ptr(), code, ldy,
          _status_ptr(dev_status, X.device))


def fp8_gated_gemm(X: torch.Tensor, sx: torch.Tensor, Wg: torch.Tensor, sg: torch.Tensor,
                   Wu: torch.Tensor, su: torch.Tensor, Q: torch.Tensor, scales: torch.Tensor,
                   dev_status: torch.Tensor | None = None) -> None:
    """Q, scales = silu(X Wg^T) * (X Wu^T) as e4m3 [m, n] with one scale per row and 128 columns;
    X as in fp8_gemm, Wg and Wu [n, k] as its W."""
    m, k = _shape2(X, "X")
    n = _shape2(Wg, "Wg")[0]
    g, gn = -(-k // 128), -(-n // 128)
    ldx, ldsx = _e4m3(X, "X", m, k), _scales(sx, "sx", m, g)
    ldg, ldsg = _e4m3(Wg, "Wg", n, k), _scales(sg, "sg", gn, g)
    ldu, ldsu = _e4m3(Wu, "Wu", n, k), _scales(su, "su", gn, g)
    ldq, lds = _e4m3(Q, "Q", m, n), _scales(scales, "scales", m, gn)
    _call(_lib.fp8_gated_gemm, "fp8_gated_gemm", X.device, (sx, Wg, sg, Wu, su, Q, scales),
          X.data_ptr(), ldx, sx.data_ptr(), ldsx, Wg.data_ptr(), ldg, sg.data_ptr(), ldsg,
          Wu.data_ptr(), ldu, su.data_ptr(), ldsu, m, n, k, Q.data_ptr(), ldq, scales.data_ptr(),
          lds, _status_ptr(dev_status, X.device))
