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
_quantize, _add_rmsnorm = _lib.fp8_quantize, _lib.fp8_add_rmsnorm
_gemm, _gated_gemm = _lib.fp8_gemm, _lib.fp8_gated_gemm
_raw_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

_DTYPES = {torch.bfloat16: GPTQ_BF16, torch.float32: GPTQ_F32, torch.float16: GPTQ_F16}
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_F32 = torch.float32
_BLOCK_ROWS = (1, 128)


def _device(t: torch.Tensor, name: str) -> int:
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _matrix(t: torch.Tensor, name: str, dev: int, rows: int, cols: int, pitch: int = 1) -> int:
    """The leading dimension of t, a [rows, cols] tensor of device `dev` with unit stride along its
    rows. One row alone has no pitch: it counts as the next multiple of `pitch`."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, is on {t.device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its last dim")
    return ld if rows > 1 else -(-cols // pitch) * pitch


def _e4m3(t: torch.Tensor, name: str, dev: int, rows: int, cols: int) -> int:
    if t.dtype not in _E4M3:
        raise ValueError(f"{name} must be float8_e4m3fn or uint8, got {t.dtype}")
    return _matrix(t, name, dev, rows, cols, 16)


def _scales(t: torch.Tensor, name: str, dev: int, rows: int, cols: int) -> int:
    if t.dtype is not torch.float32:
        raise ValueError(f"{name} must be torch.float32, got {t.dtype}")
    return _matrix(t, name, dev, rows, cols)


def _float_code(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _shape2(t: torch.Tensor, name: str) -> tuple[int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor of 2 dims")
    return t.shape


def _status_ptr(t: torch.Tensor | None, dev: int):
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not torch.int32 or t.numel() < 2 \
            or not t.is_contiguous():
        raise ValueError("dev_status must be a contiguous int32 CUDA tensor of 2 entries on the "
                         "operands' device")
    return t.data_ptr()


def _run(fn, dev: int, *args) -> None:
    """fn(*args, stream): on the current stream of device `dev`, made current for the call. The raw
    stream is asked for directly: torch.cuda.current_stream() builds a Stream object each time, 4.6
    us on the host, as much as the launch itself."""
    if dev == _get_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc:
        _check(rc, fn.__name__)


# Each call looks at its tensors twice at most. At first all in one expression, which holds for the
# layouts that programs have (a step of decoding is many calls of a few microseconds, and what
# is spent here is not hidden by anything); where it does not hold, one by one, which finds
# the leading dimensions of single rows and says what is wrong.

def fp8_quantize(X: torch.Tensor, Q: torch.Tensor, scales: torch.Tensor, block_rows: int = 1
                 ) -> None:
    """Q, scales = X [m, k] as e4m3 with one fp32 scale per 1 x 128 (activations) or 128 x 128
    (weights, block_rows=128) block."""
    m, k = _shape2(X, "X")
    code = _DTYPES.get(X.dtype)
    dev = X.get_device()
    ldx, ux = X.stride()
    rows, g = (m if block_rows == 1 else (m + 127) >> 7), (k + 127) >> 7
    if (block_rows in _BLOCK_ROWS and code is not None and dev >= 0
            and Q.shape == (m, k) and scales.shape == (rows, g)
            and Q.dtype in _E4M3 and scales.dtype is _F32
            and Q.get_device() == dev and scales.get_device() == dev):
        ldq, uq = Q.stride()
        lds, us = scales.stride()
        if ux == 1 and uq == 1 and us == 1 and rows > 1:
            return _run(_quantize, dev, X.data_ptr(), code, ldx, m, k, block_rows, Q.data_ptr(),
                        ldq, scales.data_ptr(), lds)
    if block_rows not in _BLOCK_ROWS:
        raise ValueError("block_rows must be 1 or 128")
    code = _float_code(X, "X")
    dev = _device(X, "X")
    ldx = _matrix(X, "X", dev, m, k, 8)
    ldq = _e4m3(Q, "Q", dev, m, k)
    lds = _scales(scales, "scales", dev, rows, g)
    _run(_quantize, dev, X.data_ptr(), code, ldx, m, k, block_rows, Q.data_ptr(), ldq,
         scales.data_ptr(), lds)


def fp8_add_rmsnorm(X: torch.Tensor, R: torch.Tensor | None, gamma: torch.Tensor, eps: float,
                    H: torch.Tensor | None, Q: torch.Tensor, scales: torch.Tensor) -> None:
    """h = X + R; H = h (may be X or R itself); Q, scales = h / sqrt(mean(h^2) + eps) * gamma as
    e4m3 with one scale per row and 128 columns. R and H may be None."""
    m, k = shape = _shape2(X, "X")
    t = X.dtype
    code, gcode = _DTYPES.get(t), _DTYPES.get(gamma.dtype)
    dev = X.get_device()
    ldx, ux = X.stride()
    g = (k + 127) >> 7
    if (R is not None and H is not None and code is not None and gcode is not None and dev >= 0
            and R.shape == shape and H.shape == shape and Q.shape == shape
            and scales.shape == (m, g) and gamma.shape == (k,)
            and R.dtype is t and H.dtype is t and Q.dtype in _E4M3 and scales.dtype is _F32
            and R.get_device() == dev and H.get_device() == dev and Q.get_device() == dev
            and scales.get_device() == dev and gamma.get_device() == dev):
        ldr, ur = R.stride()
        ldh, uh = H.stride()
        ldq, uq = Q.stride()
        lds, us = scales.stride()
        if (ux == 1 and ur == 1 and uh == 1 and uq == 1 and us == 1 and gamma.stride() == (1,)
                and m > 1):
            return _run(_add_rmsnorm, dev, X.data_ptr(), ldx, R.data_ptr(), ldr, code,
                        gamma.data_ptr(), gcode, eps, m, k, H.data_ptr(), ldh, Q.data_ptr(), ldq,
                        scales.data_ptr(), lds)
    code = _float_code(X, "X")
    gcode = _float_code(gamma, "gamma")
    dev = _device(X, "X")
    ldx = _matrix(X, "X", dev, m, k, 8)
    if gamma.get_device() != dev or gamma.shape != (k,) or not gamma.is_contiguous():
        raise ValueError(f"gamma must be a contiguous CUDA tensor of {k} entries on device {dev}")
    r_ptr = h_ptr = None
    ldr = ldh = 0
    if R is not None:
        if R.dtype is not X.dtype:
            raise ValueError("R must have X's dtype")
        ldr = _matrix(R, "R", dev, m, k, 8)
        r_ptr = R.data_ptr()
    if H is not None:
        if H.dtype is not X.dtype:
            raise ValueError("H must have X's dtype")
        ldh = _matrix(H, "H", dev, m, k, 8)
        h_ptr = H.data_ptr()
    ldq = _e4m3(Q, "Q", dev, m, k)
    lds = _scales(scales, "scales", dev, m, g)
    _run(_add_rmsnorm, dev, X.data_ptr(), ldx, r_ptr, ldr, code, gamma.data_ptr(), gcode, eps, m,
         k, h_ptr, ldh, Q.data_ptr(), ldq, scales.data_ptr(), lds)


def fp8_gemm(X: torch.Tensor, sx: torch.Tensor, W: torch.Tensor, sw: torch.Tensor,
             Y: torch.Tensor, dev_status: torch.Tensor | None = None) -> None:
    """Y [m, n] (bf16, fp16 or fp32) = X W^T of X [m, k] (blocks of 1 x 128, scales sx) and W [n, k]
    (blocks of 128 x 128, scales sw)."""
    m, k = _shape2(X, "X")
    n, kw = _shape2(W, "W")
    g = (k + 127) >> 7
    code = _DTYPES.get(Y.dtype)
    dev = X.get_device()
    ldx, ux = X.stride()
    ldw, uw = W.stride()
    if (kw == k and code is not None and dev >= 0 and dev_status is None
            and sx.shape == (m, g) and sw.shape == ((n + 127) >> 7, g) and Y.shape == (m, n)
            and X.dtype in _E4M3 and W.dtype in _E4M3 and sx.dtype is _F32 and sw.dtype is _F32
            and sx.get_device() == dev and W.get_device() == dev and sw.get_device() == dev
            and Y.get_device() == dev):
        ldsx, usx = sx.stride()
        ldsw, usw = sw.stride()
        ldy, uy = Y.stride()
        # a row alone has no pitch, but is as good as any other where its stride is one
        if (ux == 1 and uw == 1 and usx == 1 and usw == 1 and uy == 1 and n > 1
                and (m > 1 or (ldx >= k and ldx % 16 == 0 and ldsx >= g and ldy >= n))
                and ldsw >= g):
            return _run(_gemm, dev, X.data_ptr(), ldx, sx.data_ptr(), ldsx, W.data_ptr(), ldw,
                        sw.data_ptr(), ldsw, m, n, k, Y.data_ptr(), code, ldy, None)
    dev = _device(X, "X")
    ldx, ldsx = _e4m3(X, "X", dev, m, k), _scales(sx, "sx", dev, m, g)
    ldw, ldsw = _e4m3(W, "W", dev, n, k), _scales(sw, "sw", dev, -(-n // 128), g)
    code = _float_code(Y, "Y")
    ldy = _matrix(Y, "Y", dev, m, n, 8)
    _run(_gemm, dev, X.data_ptr(), ldx, sx.data_ptr(), ldsx, W.data_ptr(), ldw, sw.data_ptr(), ldsw,
         m, n, k, Y.data_ptr(), code, ldy, _status_ptr(dev_status, dev))


def fp8_gated_gemm(X: torch.Tensor, sx: torch.Tensor, Wg: torch.Tensor, sg: torch.Tensor,
                   Wu: torch.Tensor, su: torch.Tensor, Q: torch.Tensor, scales: torch.Tensor,
                   dev_status: torch.Tensor | None = None) -> None:
    """Q, scales = silu(X Wg^T) * (X Wu^T) as e4m3 [m, n] with one scale per row and 128 columns;
    X as in fp8_gemm, Wg and Wu [n, k] as its W."""
    m, k = _shape2(X, "X")
    n = _shape2(Wg, "Wg")[0]
    g, gn = -(-k // 128), -(-n // 128)
    dev = _device(X, "X")
    ldx, ldsx = _e4m3(X, "X", dev, m, k), _scales(sx, "sx", dev, m, g)
    ldg, ldsg = _e4m3(Wg, "Wg", dev, n, k), _scales(sg, "sg", dev, gn, g)
    ldu, ldsu = _e4m3(Wu, "Wu", dev, n, k), _scales(su, "su", dev, gn, g)
    ldq, lds = _e4m3(Q, "Q", dev, m, n), _scales(scales, "scales", dev, m, gn)
    _run(_gated_gemm, dev, X.data_ptr(), ldx, sx.data_ptr(), ldsx, Wg.data_ptr(), ldg,
         sg.data_ptr(), ldsg, Wu.data_ptr(), ldu, su.data_ptr(), ldsu, m, n, k, Q.data_ptr(), ldq,
         scales.data_ptr(), lds, _status_ptr(dev_status, dev))
