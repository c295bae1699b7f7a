"""The e4m3 format with one fp32 scale per block of 128, and the operators on it.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0 is subnormal (step 2^-9), the
code 0x7F (and 0xFF) is NaN, there are no infinities, the largest value is 448.

The scale of a block and the code of an element are decisions of fp32 arithmetic, as in the
quantizer of the integer formats: s = fl(amax / 448), code = e4m3(fl(y * fl(1 / s))) in fp32 with
round-to-nearest-even. Everything else is float64.

Pinned by: the table written out from the definition against hand values; the encoder against
torch's conversion on every fp16 value; the products against brute-force loops.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_SCALE = np.float32(2.0 ** -126)


def table() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1.0 + f / 8.0) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            v = np.nan
        out[c] = -v if c & 0x80 else v
    return out


_POS = table()[:127]                       # 0 .. 448, ascending with the code
_MID = (_POS[1:] + _POS[:-1]) / 2.0        # exact: one more bit than a value


def encode(v: np.ndarray) -> np.ndarray:
    """Codes of v: nearest, ties to the even code, +-448 beyond, NaN for NaN."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    lo = np.searchsorted(_MID, a, side="left")           # ties: the lower code
    tie = (lo < 126) & (a == _MID[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = code | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    return table()[np.asarray(codes, np.uint8)]


def spread(S: np.ndarray, rows: int, m: int, k: int) -> np.ndarray:
    """The scale of every element of an [m, k] matrix."""
    return np.repeat(np.repeat(S, rows, axis=0)[:m], 128, axis=1)[:, :k]


def block_max(Y: np.ndarray, rows: int) -> np.ndarray:
    """The largest magnitude of each block of rows x 128; NaN where a block is not finite."""
    m, k = Y.shape
    out = np.zeros((-(-m // rows), -(-k // 128)), Y.dtype)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            b = np.abs(Y[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128])
            out[i, j] = b.max() if np.isfinite(b).all() else np.nan
    return out


def scales_of(amax: np.ndarray) -> np.ndarray:
    """fp32 scales from fp32 maxima."""
    a = np.asarray(amax, np.float32)
    s = np.maximum(a / np.float32(E4M3_MAX), MIN_SCALE)
    return np.where(a == 0, np.float32(1), s).astype(np.float32)


def quantize(Y: np.ndarray, rows: int) -> tuple[np.ndarray, np.ndarray]:
    """(codes, scales) of an fp32 matrix."""
    Y = np.asarray(Y, np.float32)
    S = scales_of(block_max(Y, rows))
    with np.errstate(invalid="ignore"):
        inv = (np.float32(1) / S).astype(np.float32)
        v = Y * spread(inv, rows, *Y.shape)
    return encode(v), S


def dequantize(codes: np.ndarray, S: np.ndarray, rows: int) -> np.ndarray:
    return decode(codes) * spread(np.asarray(S, np.float64), rows, *codes.shape)


def add_rmsnorm(X, R, gamma, eps: float) -> tuple[np.ndarray, np.ndarray]:
    """(h, y) in float64."""
    h = np.asarray(X, np.float64) if R is None else np.asarray(X, np.float64) + R
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    return h, y


def gemm(cx, sx, cw, sw) -> tuple[np.ndarray, np.ndarray]:
    """(Y, sum of the terms' magnitudes) in float64."""
    x, w = dequantize(cx, sx, 1), dequantize(cw, sw, 128)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def silu(g: np.ndarray) -> np.ndarray:
    return g / (1.0 + np.exp(-np.clip(g, -700.0, None)))
