"""Shared by the GPU tests of the e4m3 operators: buffers with guard values, error bounds."""
import numpy as np
import torch

from oracle import fp8 as o

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a step of a rounding, relative to the value (u of the type)
HALF_STEP = {t: torch.finfo(d).eps / 2 for t, d in DTYPES.items()}


def padded(m, k, dtype, ld=None, fill=0x7F, offset=0):
    """An [m, k] view of a flat buffer whose other bytes hold `fill` (e4m3 NaN), and the buffer."""
    ld = k if ld is None else ld
    size = torch.empty(0, dtype=dtype).element_size()
    n = (m * ld + offset) * size
    raw = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
    return raw[:n].view(dtype)[offset:].view(m, ld)[:, :k], raw


def untouched(raw, view, fill=0x7F):
    """Every byte of the buffer outside the view still holds the fill value."""
    keep = torch.ones(raw.numel(), dtype=torch.bool, device=raw.device)
    size = view.element_size()
    at = (view.data_ptr() - raw.data_ptr()) + size * (
        torch.arange(view.shape[0], device=raw.device)[:, None] * view.stride(0)
        + torch.arange(view.shape[1], device=raw.device)[None, :])
    for b in range(size):
        keep[(at + b).reshape(-1)] = False
    return bool((raw[keep] == fill).all())


def codes_of(q):
    return q.contiguous().view(torch.uint8).cpu().numpy()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_format(codes, S, y, dy, rows=1):
    """codes and S hold y [m, k] (float64, each element known within dy): every block's scale is
    amax / 448 within the block's largest dy and one fp32 rounding, and every code is the rounding
    of some value within dy, given the scale."""
    m, k = y.shape
    amax = o.block_max(np.abs(y), rows)
    slack = o.block_max(np.broadcast_to(dy, y.shape), rows) / 448 + 2.0 ** -23 * amax / 448
    want = np.where(amax == 0, 1.0, np.maximum(amax / 448, 2.0 ** -126))
    assert np.array_equal(np.isnan(S), np.isnan(want))
    ok = ~np.isnan(want)
    # a block whose every element is zero within dy may be a block of zeros (fp32 underflow), scale 1
    zero = (S == 1) & (o.block_max(np.maximum(np.abs(y) - dy, 0.0), rows) == 0)
    ok &= ~zero
    assert np.all(np.abs(S[ok] - want[ok]) <= slack[ok]), np.max(np.abs(S - want)[ok] / want[ok])
    s = o.spread(S.astype(np.float64), rows, m, k)
    fine = ~np.isnan(s)
    # y * fl(1 / s): two more fp32 roundings
    d = dy + np.abs(y) * 2.0 ** -23
    v = o.decode(codes)
    lo, hi = o.decode(o.encode((y - d) / s)), o.decode(o.encode((y + d) / s))
    assert np.all((v[fine] >= lo[fine]) & (v[fine] <= hi[fine]))
    assert np.all(np.isnan(v[~fine]))


def gemm_bound(A, k):
    """|Y - Y64| before the output's rounding, A the sum of the terms' magnitudes: a block's 128
    exact products summed in fp32 in any order, each addition truncated (128 * 2^-23), then
    ceil(k / 128) blocks scaled (two roundings) and added (2^-24 each)."""
    return A * (128 * 2.0 ** -23 + (-(-k // 128) + 2) * 2.0 ** -24)
