"""Pins of the oracle of the e4m3 format: hand values, torch's conversion, brute-force loops."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as o


def test_table_hand_values():
    t = o.table()
    assert t[0x00] == 0.0 and t[0x01] == 2.0 ** -9 and t[0x07] == 7 * 2.0 ** -9
    assert t[0x08] == 2.0 ** -6                       # the smallest normal number
    assert t[0x38] == 1.0 and t[0x39] == 1.125 and t[0xB8] == -1.0
    assert t[0x7E] == 448.0 and t[0xFE] == -448.0
    assert math.isnan(t[0x7F]) and math.isnan(t[0xFF])
    assert t[0x77] == 240.0 and t[0x78] == 256.0


def test_table_matches_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    np.testing.assert_array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), o.table())


def test_encode_matches_torch_on_every_fp16_up_to_448():
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16).float()
    v = v[v.abs() <= 448]                             # ties among them: every midpoint is an fp16
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(o.encode(v.numpy()), want)


def test_encode_saturates_and_keeps_nan():
    got = o.encode(np.array([448.0, 449.0, 1e30, -1e30, np.nan]))
    assert got.tolist()[:4] == [0x7E, 0x7E, 0x7E, 0xFE] and got[4] == 0x7F


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_scales_and_step(rows):
    rng = np.random.default_rng(rows)
    Y = (rng.standard_normal((130, 300)) * np.exp(rng.standard_normal(300))).astype(np.float32)
    codes, S = o.quantize(Y, rows)
    assert S.shape == (130 if rows == 1 else 2, 3) and S.dtype == np.float32
    b = Y[:rows, :128]
    assert S[0, 0] == np.float32(np.abs(b).max()) / np.float32(448)
    # each element is off by at most half a step: 2^-4 of it, or half a subnormal step
    back = o.dequantize(codes, S, rows)
    step = np.maximum(np.abs(Y) * 2.0 ** -4, o.spread(S, rows, *Y.shape) * 2.0 ** -10)
    assert np.all(np.abs(back - Y) <= step * (1 + 2.0 ** -20))
    # the largest value of a block becomes +-448
    assert np.all(o.block_max(o.decode(codes), rows) == 448)


def test_quantize_degenerate_blocks():
    Y = np.zeros((2, 256), np.float32)
    Y[0, 3] = np.float32(2.0 ** -140)                 # 1 / (amax / 448) would overflow
    Y[1, 200] = np.inf
    codes, S = o.quantize(Y, 1)
    assert S[0, 0] == np.float32(2.0 ** -126) and S[0, 1] == 1 and S[1, 0] == 1
    assert np.isnan(S[1, 1]) and np.all(codes[1, 128:] == 0x7F) and np.all(codes[1, :128] == 0)


def test_gemm_against_loops():
    rng = np.random.default_rng(3)
    m, n, k = 3, 130, 150
    cx, sx = o.quantize(rng.standard_normal((m, k)), 1)
    cw, sw = o.quantize(rng.standard_normal((n, k)), 128)
    Y, A = o.gemm(cx, sx, cw, sw)
    t = o.table()
    for i, j in [(0, 0), (2, 129), (1, 127), (1, 128)]:
        terms = [t[cx[i, c]] * float(sx[i, c // 128]) * t[cw[j, c]] * float(sw[j // 128, c // 128])
                 for c in range(k)]
        assert abs(Y[i, j] - math.fsum(terms)) <= 1e-13 * A[i, j]
        assert abs(A[i, j] - math.fsum(abs(x) for x in terms)) <= 1e-13 * A[i, j]


def test_norm_hand_case():
    h, y = o.add_rmsnorm(np.array([[1.0, 2.0]]), np.array([[2.0, 2.0]]), np.array([1.0, 0.5]), 0.0)
    r = math.sqrt(12.5)
    np.testing.assert_allclose(h, [[3.0, 4.0]], rtol=0)
    np.testing.assert_allclose(y, [[3.0 / r, 2.0 / r]], rtol=1e-15)
    assert o.silu(np.array([0.0, -1000.0, 1000.0])).tolist() == [0.0, -1000.0 * math.exp(-700), 1000.0]
