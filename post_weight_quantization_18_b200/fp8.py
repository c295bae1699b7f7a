"""Layers held in e4m3 with one fp32 scale per block of 128: allocation over the C ABI's calls.

    w = fp8.quantize_weight(W)                       # [n, k] bf16, fp16 or fp32 -> FP8Matrix
    x = fp8.quantize_activations(X)                  # [m, k] -> FP8Matrix
    Y = fp8.linear(x, w)                             # [m, n] bf16
    mlp = fp8.GatedMLP.from_weights(gamma, Wg, Wu, Wd)
    y, h = mlp(X, residual)                          # norm -> gated pair -> down projection

As in `layer`, all arithmetic runs in the library's kernels; this module only sizes and allocates
buffers and orders the calls on the current stream.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _fp8 as F


@dataclass
class FP8Matrix:
    q: torch.Tensor            # float8_e4m3fn [m, k], rows a multiple of 16 bytes apart
    scales: torch.Tensor       # fp32 [ceil(m / block_rows), ceil(k / 128)]
    block_rows: int            # 1 (activations) or 128 (weights)

    @property
    def shape(self):
        return self.q.shape

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The values as a dense matrix (for inspection; not a path of the products)."""
        m, k = self.q.shape
        s = self.scales.repeat_interleave(self.block_rows, 0)[:m].repeat_interleave(128, 1)[:, :k]
        return (self.q.float() * s).to(dtype)


def empty(m: int, k: int, block_rows: int = 1, device="cuda") -> FP8Matrix:
    """An uninitialised matrix of the format, laid out for the tensor cores."""
    ld = -(-k // 16) * 16
    q = torch.empty((m, ld), dtype=torch.float8_e4m3fn, device=device)[:, :k]
    s = torch.empty((-(-m // block_rows), -(-k // 128)), dtype=torch.float32, device=device)
    return FP8Matrix(q, s, block_rows)


def _quantize(X: torch.Tensor, block_rows: int) -> FP8Matrix:
    out = empty(X.shape[0], X.shape[1], block_rows, X.device)
    F.fp8_quantize(X, out.q, out.scales, block_rows)
    return out


def quantize_weight(W: torch.Tensor) -> FP8Matrix:
    """W [n, k] in blocks of 128 x 128."""
    return _quantize(W, 128)


def quantize_activations(X: torch.Tensor) -> FP8Matrix:
    """X [m, k] in blocks of 1 x 128."""
    return _quantize(X, 1)


def _want(x: FP8Matrix, block_rows: int, name: str) -> None:
    if x.block_rows != block_rows:
        raise ValueError(f"{name} must hold blocks of {block_rows} x 128")


def add_rmsnorm(X: torch.Tensor, residual: torch.Tensor | None, gamma: torch.Tensor,
                eps: float = 1e-5) -> tuple[FP8Matrix, torch.Tensor]:
    """(the norm of h in the format, h) for h = X + residual."""
    out = empty(X.shape[0], X.shape[1], 1, X.device)
    H = X if residual is None else torch.empty_like(X, memory_format=torch.contiguous_format)
    F.fp8_add_rmsnorm(X, residual, gamma, eps, None if residual is None else H, out.q, out.scales)
    return out, H


def linear(x: FP8Matrix, w: FP8Matrix, dtype: torch.dtype = torch.bfloat16,
           dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """Y [m, n] = x w^T."""
    _want(x, 1, "x")
    _want(w, 128, "w")
    Y = torch.empty((x.shape[0], w.shape[0]), dtype=dtype, device=x.q.device)
    F.fp8_gemm(x.q, x.scales, w.q, w.scales, Y, dev_status)
    return Y


def gated(x: FP8Matrix, wg: FP8Matrix, wu: FP8Matrix,
          dev_status: torch.Tensor | None = None) -> FP8Matrix:
    """silu(x wg^T) * (x wu^T) in the format."""
    _want(x, 1, "x")
    _want(wg, 128, "wg")
    _want(wu, 128, "wu")
    out = empty(x.shape[0], wg.shape[0], 1, x.q.device)
    F.fp8_gated_gemm(x.q, x.scales, wg.q, wg.scales, wu.q, wu.scales, out.q, out.scales,
                     dev_status)
    return out


@dataclass
class GatedMLP:
    """The feed-forward half of a decoder block on e4m3 weights."""
    gamma: torch.Tensor
    gate: FP8Matrix
    up: FP8Matrix
    down: FP8Matrix
    eps: float = 1e-5

    @classmethod
    def from_weights(cls, gamma: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                     Wd: torch.Tensor, eps: float = 1e-5) -> "GatedMLP":
        return cls(gamma, quantize_weight(Wg), quantize_weight(Wu), quantize_weight(Wd), eps)

    def __call__(self, X: torch.Tensor, residual: torch.Tensor | None = None,
                 dev_status: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """(down projection's output, h = X + residual); the next norm adds the two."""
        x, h = add_rmsnorm(X, residual, self.gamma, self.eps)
        hidden = gated(x, self.gate, self.up, dev_status)
        return linear(hidden, self.down, X.dtype, dev_status), h
