"""GPU parity of fp8_quantize and fp8_add_rmsnorm with the float64 oracle.

fp8_quantize takes its decisions in fp32 exactly as the oracle does (maximum, division by 448,
reciprocal, product, rounding), so codes and scales are compared bit for bit. The norm sums squares
in another order than the oracle; its y is known within NORM_REL of itself:
  the sum of k squares: at most 40 additions in a row per thread, 10 in the tree, 2^-24 each, halved
  by the square root (25 * 2^-24); h, the division by k, + eps, sqrt, reciprocal, two products: one
  rounding each, of which those under the root count half (6 * 2^-24). 31 * 2^-24 < 2^-19.
"""
import numpy as np
import pytest
import torch

from fp8_util import DTYPES, HALF_STEP, check_format, codes_of, f64, padded, untouched
from oracle import fp8 as o

pytestmark = pytest.mark.gpu

NORM_REL = 2.0 ** -19


def _values(m, k, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g) * torch.exp(torch.randn(k, generator=g))
    return x.to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,k", [
    (1, 1), (1, 128), (3, 127), (2, 129), (129, 8), (128, 256), (5, 1000), (130, 645), (257, 2184),
])
def test_quantize_equals_oracle(dtype, rows, m, k):
    import post_weight_quantization_18_b200 as G
    X = _values(m, k, m * 1000 + k, dtype)
    X[m // 2, : k // 3] = 0                               # a block of zeros where k allows one
    Q, raw_q = padded(m, k, torch.uint8, ld=-(-k // 16) * 16)
    S, raw_s = padded(-(-m // rows), -(-k // 128), torch.float32, ld=-(-k // 128) + 3)
    G.fp8_quantize(X.cuda(), Q, S, rows)
    codes, scales = o.quantize(X.float().numpy(), rows)
    np.testing.assert_array_equal(S.cpu().numpy(), scales)
    np.testing.assert_array_equal(codes_of(Q), codes)
    assert untouched(raw_q, Q) and untouched(raw_s, S)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("off,ldx,ldq,offq", [(1, 301, 303, 3), (0, 304, 301, 0), (8, 320, 312, 8)])
def test_quantize_any_alignment(rows, off, ldx, ldq, offq):
    """Rows that no vector load or store can take, and columns of a wider matrix."""
    import post_weight_quantization_18_b200 as G
    m, k = 40, 300
    X, _ = padded(m, k, torch.bfloat16, ld=ldx, offset=off)
    X.copy_(_values(m, k, 5, "bf16"))
    Q, raw_q = padded(m, k, torch.uint8, ld=ldq, offset=offq)
    S = torch.full((-(-m // rows), 3), -1.0, device="cuda")
    G.fp8_quantize(X, Q.view(torch.float8_e4m3fn), S, rows)
    codes, scales = o.quantize(X.float().cpu().numpy(), rows)
    np.testing.assert_array_equal(S.cpu().numpy(), scales)
    np.testing.assert_array_equal(codes_of(Q), codes)
    assert untouched(raw_q, Q)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_degenerate_and_nonfinite_blocks(rows):
    import post_weight_quantization_18_b200 as G
    X = _values(256, 512, 9, "fp32")
    X[0, :128] = 0
    X[0, 5] = 2.0 ** -140                                 # subnormal: 1 / (amax / 448) overflows
    X[1, 130] = float("nan")
    X[2, 300] = float("inf")
    X[3, 400] = -float("inf")
    X[200, :] = 3e38                                      # the largest scales
    if rows == 128:
        X[:128, 128:256] = X[:128, 128:256].nan_to_num(0)
        X[130, 140] = float("nan")
        X[:128, :128] = 0
        X[7, 9] = -2.0 ** -149
    Q = torch.empty((256, 512), dtype=torch.float8_e4m3fn, device="cuda")
    S = torch.empty((256 // rows, 4), device="cuda")
    G.fp8_quantize(X.cuda(), Q, S, rows)
    codes, scales = o.quantize(X.numpy(), rows)
    np.testing.assert_array_equal(S.cpu().numpy(), scales)
    np.testing.assert_array_equal(codes_of(Q) & 0x7F, codes & 0x7F)
    nan = np.isnan(o.spread(scales, rows, 256, 512))
    np.testing.assert_array_equal(codes_of(Q)[~nan], codes[~nan])
    assert np.isnan(scales).any() and (scales == np.float32(2.0 ** -126)).any()


def test_quantize_ties_and_subnormal_codes():
    """A block whose scale is exactly 1: midpoints of neighbouring codes go to the even one."""
    import post_weight_quantization_18_b200 as G
    mids = (o.table()[1:127] + o.table()[:126]) / 2
    X = torch.zeros((2, 128))
    X[0, :126] = torch.from_numpy(mids).float()
    X[1] = -X[0]
    X[:, 127] = 448.0
    Q = torch.empty((2, 128), dtype=torch.uint8, device="cuda")
    S = torch.empty((2, 1), device="cuda")
    G.fp8_quantize(X.cuda(), Q, S)
    assert S.cpu().tolist() == [[1.0], [1.0]]
    np.testing.assert_array_equal(Q.cpu().numpy(), o.encode(X.numpy()))


def _norm_case(m, k, dtype, gdtype, seed, with_r=True):
    X, R = _values(m, k, seed, dtype), _values(m, k, seed + 1, dtype)
    gamma = (1 + 0.3 * torch.randn(k, generator=torch.Generator().manual_seed(seed + 2)))
    return X, (R if with_r else None), gamma.to(DTYPES[gdtype])


def _check_norm(X, R, gamma, eps, H, Q, S, dtype):
    h, y = o.add_rmsnorm(f64(X), None if R is None else f64(R), f64(gamma), eps)
    # h = x + r is formed in fp32: where x and r cancel, y is off by that rounding of h
    dh = 0.0 if R is None else np.abs(h) * 2.0 ** -24
    check_format(codes_of(Q), S.cpu().numpy(), y, np.abs(y) * NORM_REL)
    if H is not None:
        u = HALF_STEP[dtype]
        tiny = 2.0 ** -25 if dtype == "fp16" else 0.0      # half a subnormal step of fp16
        assert np.all(np.abs(f64(H) - h) <= np.maximum(np.abs(h) * u * (1 + 2.0 ** -12), tiny) + dh)


@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                          ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("m,k", [
    (1, 1), (2, 8), (3, 127), (4, 129), (33, 1000), (5, 4096), (3, 4104), (7, 5120), (2, 8200),
    (2, 11800), (3, 12288), (3, 16384), (2, 16392), (2, 40007),                   # one, two, four vectors; the long rows
])
def test_norm_matches_oracle(dtype, gdtype, m, k):
    import post_weight_quantization_18_b200 as G
    X, R, gamma = _norm_case(m, k, dtype, gdtype, k + m)
    H, raw_h = padded(m, k, DTYPES[dtype], ld=k + 8)
    Q, raw_q = padded(m, k, torch.uint8, ld=-(-k // 16) * 16)
    S, raw_s = padded(m, -(-k // 128), torch.float32, ld=-(-k // 128) + 1)
    G.fp8_add_rmsnorm(X.cuda(), R.cuda(), gamma.cuda(), 1e-5, H, Q, S)
    _check_norm(X, R, gamma, np.float32(1e-5), H, Q, S, dtype)
    assert untouched(raw_h, H) and untouched(raw_q, Q) and untouched(raw_s, S)


@pytest.mark.parametrize("k", [1000, 2500])
def test_norm_without_residual_and_in_place(k):
    import post_weight_quantization_18_b200 as G
    m = 37
    X, R, gamma = _norm_case(m, k, "bf16", "bf16", 3)
    Q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    S = torch.empty((m, -(-k // 128)), device="cuda")
    G.fp8_add_rmsnorm(X.cuda(), None, gamma.cuda(), 1e-6, None, Q, S)
    _check_norm(X, None, gamma, np.float32(1e-6), None, Q, S, "bf16")
    H0 = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    Q0, S0 = torch.empty_like(Q), torch.empty_like(S)
    G.fp8_add_rmsnorm(X.cuda(), R.cuda(), gamma.cuda(), 1e-6, H0, Q0, S0)
    for which in range(2):                                # H is X, H is R
        x, r = X.cuda(), R.cuda()
        h = (x, r)[which]
        G.fp8_add_rmsnorm(x, r, gamma.cuda(), 1e-6, h, Q, S)
        assert torch.equal(h, H0) and torch.equal(Q, Q0) and torch.equal(S, S0)


def test_norm_in_place_on_long_rows():
    import post_weight_quantization_18_b200 as G
    m, k = 2, 20000
    X, R, gamma = _norm_case(m, k, "bf16", "bf16", 4)
    Q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    S = torch.empty((m, -(-k // 128)), device="cuda")
    r = R.cuda()
    G.fp8_add_rmsnorm(X.cuda(), r, gamma.cuda(), 1e-6, r, Q, S)
    _check_norm(X, R, gamma, np.float32(1e-6), r, Q, S, "bf16")


@pytest.mark.parametrize("off,ld", [(1, 1001), (0, 1003), (4, 1004)])
def test_norm_any_alignment(off, ld):
    import post_weight_quantization_18_b200 as G
    m, k = 9, 1000
    X, R, gamma = _norm_case(m, k, "bf16", "bf16", 6)
    x, _ = padded(m, k, torch.bfloat16, ld=ld, offset=off)
    x.copy_(X)
    g, _ = padded(1, k, torch.bfloat16, offset=off)
    g.copy_(gamma[None])
    H, raw_h = padded(m, k, torch.bfloat16, ld=ld, offset=off)
    Q, raw_q = padded(m, k, torch.uint8, ld=ld, offset=off)
    S = torch.empty((m, 8), device="cuda")
    G.fp8_add_rmsnorm(x, R.cuda(), g[0], 1e-5, H, Q, S)
    _check_norm(X, R, gamma, np.float32(1e-5), H, Q, S, "bf16")
    assert untouched(raw_h, H) and untouched(raw_q, Q)


@pytest.mark.parametrize("off,ld", [(0, 1004), (4, 1008), (8, 1000), (2, 1002), (1, 1001)])
@pytest.mark.parametrize("k", [1000, 997])
def test_fp32_rows_of_any_alignment(off, ld, k):
    """Rows that start at 4, 8, 16 or 32 bytes, or at these in turn."""
    import post_weight_quantization_18_b200 as G
    m = 9
    X, R, gamma = _norm_case(m, k, "fp32", "fp32", 6)
    x, _ = padded(m, k, torch.float32, ld=ld, offset=off)
    x.copy_(X)
    H, raw_h = padded(m, k, torch.float32, ld=ld, offset=off)
    Q, raw_q = padded(m, k, torch.uint8, ld=1008)
    S = torch.empty((m, 8), device="cuda")
    G.fp8_add_rmsnorm(x, R.cuda(), gamma.cuda(), 1e-5, H, Q, S)
    _check_norm(X, R, gamma, np.float32(1e-5), H, Q, S, "fp32")
    assert untouched(raw_h, H) and untouched(raw_q, Q)
    for rows in (1, 128):
        S = torch.empty((-(-m // rows), 8), device="cuda")
        G.fp8_quantize(x, Q, S, rows)
        codes, scales = o.quantize(X.numpy(), rows)
        np.testing.assert_array_equal(S.cpu().numpy(), scales)
        np.testing.assert_array_equal(codes_of(Q), codes)
    assert untouched(raw_q, Q)


def test_norm_zero_rows_and_nonfinite():
    """A row of zeros: y = 0, scales 1. With eps = 0 it is 0 / 0, as the formula says. A NaN or an
    infinity makes NaN what it reaches and leaves the other rows alone."""
    import post_weight_quantization_18_b200 as G
    m, k = 4, 512
    X = _values(m, k, 8, "fp32")
    X[0] = 0
    X[1, 7] = float("nan")
    X[2, 300] = float("inf")
    gamma = torch.ones(k)
    Q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    S = torch.empty((m, 4), device="cuda")
    G.fp8_add_rmsnorm(X.cuda(), None, gamma.cuda(), 1e-5, None, Q, S)
    s, q = S.cpu(), Q.cpu()
    assert s[0].tolist() == [1.0] * 4 and not q[0].any()
    assert torch.isnan(s[1]).all() and ((q[1] & 0x7F) == 0x7F).all()
    # row 2: 1 / sqrt(inf) = 0; inf * 0 is NaN in its block, the finite elements become 0
    assert torch.isnan(s[2]).tolist() == [False, False, True, False]
    assert ((q[2, 256:384] & 0x7F) == 0x7F).all() and not (q[2, :256] & 0x7F).any()
    _check_norm(X[3:], None, gamma, np.float32(1e-5), None, Q[3:], S[3:], "fp32")
    G.fp8_add_rmsnorm(X.cuda(), None, gamma.cuda(), 0.0, None, Q, S)
    assert torch.isnan(S[0]).all() and not torch.isnan(S[3]).any()


def test_zero_rows_are_a_call():
    import post_weight_quantization_18_b200 as G
    X = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    Q = torch.empty((0, 256), dtype=torch.float8_e4m3fn, device="cuda")
    S = torch.empty((0, 2), device="cuda")
    for rows in (1, 128):
        G.fp8_quantize(X, Q, S, rows)
    G.fp8_add_rmsnorm(X, X, torch.ones(256, device="cuda"), 1e-5, X, Q, S)


def test_quantize_offsets_past_32_bits():
    """A matrix of more than 2^32 bytes, of which the last rows are looked at."""
    import post_weight_quantization_18_b200 as G
    m, k = 140_000, 16_384                                # 2.3e9 elements
    X = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    X[-130:] = _values(130, k, 12, "bf16").cuda()
    for rows in (1, 128):
        out = G.fp8.empty(m, k, rows)
        G.fp8_quantize(X, out.q, out.scales, rows)
        keep = 130 if rows == 1 else 128 + m % 128        # whole blocks at the end
        first = m - keep if rows == 1 else m // 128 * 128 - 128
        tail = X[first:].float().cpu().numpy()
        codes, scales = o.quantize(tail, rows)
        np.testing.assert_array_equal(codes_of(out.q[first:]), codes)
        np.testing.assert_array_equal(out.scales[-scales.shape[0]:].cpu().numpy(), scales)
        assert not out.q[:first].view(torch.uint8).any() or rows == 128
        del out


def test_binding_refuses_mixed_tensors():
    import post_weight_quantization_18_b200 as G
    X = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros((4, 256), dtype=torch.uint8, device="cuda")
    S = torch.zeros((4, 2), device="cuda")
    g = torch.ones(256, device="cuda")
    with pytest.raises(ValueError, match=r"Q must be \[4, 256\]"):
        G.fp8_quantize(X, Q[:, :255], S)
    with pytest.raises(ValueError, match=r"scales must be \[1, 2\]"):
        G.fp8_quantize(X, Q, S, 128)
    with pytest.raises(ValueError, match="unit stride"):
        G.fp8_quantize(torch.zeros((256, 4), dtype=torch.bfloat16, device="cuda").t(), Q, S)
    with pytest.raises(ValueError, match="CUDA"):
        G.fp8_quantize(X, Q.cpu(), S)
    with pytest.raises(ValueError, match="X's dtype"):
        G.fp8_add_rmsnorm(X, X.float(), g, 1e-5, None, Q, S)
    with pytest.raises(ValueError, match="gamma"):
        G.fp8_add_rmsnorm(X, None, g[:255], 1e-5, None, Q, S)
    with pytest.raises(G.GPTQError) as e:                 # fp16 gamma on bf16 rows
        G.fp8_add_rmsnorm(X, None, g.half(), 1e-5, None, Q, S)
    assert e.value.code == 2
    with pytest.raises(G.GPTQError) as e:                 # rows that overlap
        G.fp8_quantize(X[:1].expand(4, 256), Q, S)
    assert e.value.code == 1


# (width, what takes it): a warp a row with one and two vectors, a CTA with one, two and four, long rows.
NORM_FORMS = [200, 500, 2048, 5120, 12288, 20000]


def _check_norm_small(X, gamma, eps, Q, S):
    """As _check_norm, with the spacing of subnormal numbers: h / rms is off by half of it, times gamma,
    and y by another half."""
    g = f64(gamma)
    _, y = o.add_rmsnorm(f64(X), None, g, eps)
    dy = np.abs(y) * NORM_REL + 2.0 ** -150 * (1 + np.abs(g))
    check_format(codes_of(Q), S.cpu().numpy(), y, dy)


@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("k", NORM_FORMS)
def test_norm_blocks_of_very_small_values(k, dtype, gdtype):
    """Zeros beside values for which 1 / s is large, at a 1 / rms of 1 to 316: every scale is finite, so no
    code may be NaN, and the zeros stay zeros."""
    import post_weight_quantization_18_b200 as G
    m = 4
    X = _values(m, k, k, dtype)
    X[0, :128] = 0
    X[0, 3], X[0, 4] = 1e-36, 5e-37                       # in a row of ordinary values
    X[1] = 0
    X[1, ::3] = 1e-37                                     # a whole row: 1 / rms = 1 / sqrt(eps)
    X[1, 1::7] = -3e-38
    X[2] = (X[2].float() * 0.01).to(X.dtype)
    X[2, 128:] = 0
    X[2, 130::5] = 2.0 ** -130                            # subnormal in every type here
    gamma = torch.ones(k).to(DTYPES[gdtype])
    Q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    S = torch.empty((m, -(-k // 128)), device="cuda")
    G.fp8_add_rmsnorm(X.cuda(), None, gamma.cuda(), 1e-5, None, Q, S)
    assert torch.isfinite(S).all() and not ((Q & 0x7F) == 0x7F).any()
    assert not (Q.cpu()[X == 0] & 0x7F).any()
    _check_norm_small(X, gamma, np.float32(1e-5), Q, S)


@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("k", NORM_FORMS)
def test_norm_takes_gamma_after_the_mean(k, dtype, gdtype):
    """y is an ordinary number although h gamma is none: gamma beyond 1e19 with large h, far below 1 with
    small h. bf16 and fp32 rows of all sizes; of fp16 the ordinary ones."""
    import post_weight_quantization_18_b200 as G
    size = (1.0, 1.0, 1.0) if dtype == "fp16" else (1e16, 1.0, 1e-18)
    m = 3
    X = _values(m, k, k + 1, "fp32").clamp(-4, 4)
    X = (X * torch.tensor(size)[:, None]).to(DTYPES[dtype])
    gamma = torch.ones(k)
    gamma[:60] = 1e25
    gamma[128:] = 1e-27
    gamma = gamma.to(DTYPES[gdtype])
    Q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    S = torch.empty((m, -(-k // 128)), device="cuda")
    G.fp8_add_rmsnorm(X.cuda(), None, gamma.cuda(), 1e-37, None, Q, S)
    assert torch.isfinite(S).all()
    _check_norm_small(X, gamma, np.float32(1e-37), Q, S)


# Rows enough that every warp or CTA of the persistent forms takes three and more, the last round ragged: a
# warp a row with one and two vectors, a CTA a row with one, two and four.
NORM_ROUNDS = [(15001, 200), (15001, 500), (4001, 2048), (1501, 5120), (1201, 12288)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k", NORM_ROUNDS)
def test_norm_over_many_rounds_of_rows(m, k, dtype):
    """Every row of a long call is what a call of few rows, each in its first round, makes of it; and some
    rows of the first, a middle and the last round against the oracle."""
    import post_weight_quantization_18_b200 as G
    X, R, gamma = _norm_case(m, k, dtype, "fp32", 5)
    x, r, g = X.cuda(), R.cuda(), gamma.cuda()
    H, raw_h = padded(m, k, DTYPES[dtype], ld=k + 8)
    Q, raw_q = padded(m, k, torch.uint8, ld=-(-k // 16) * 16)
    S, raw_s = padded(m, -(-k // 128), torch.float32, ld=-(-k // 128) + 1)
    G.fp8_add_rmsnorm(x, r, g, 1e-5, H, Q, S)
    few = 144
    for i in range(0, m, few):
        n = min(few, m - i)
        h, q, s = torch.empty_like(x[i:i + n]), torch.empty_like(Q[i:i + n]), torch.empty_like(S[i:i + n])
        G.fp8_add_rmsnorm(x[i:i + n], r[i:i + n], g, 1e-5, h, q, s)
        assert torch.equal(h, H[i:i + n]) and torch.equal(q, Q[i:i + n]) and torch.equal(s, S[i:i + n]), i
    for i in (0, m // 2, m - 8):
        _check_norm(X[i:i + 8], R[i:i + 8], gamma, np.float32(1e-5), H[i:i + 8], Q[i:i + 8], S[i:i + 8],
                    dtype)
    assert untouched(raw_h, H) and untouched(raw_q, Q) and untouched(raw_s, S)
    for which in range(2):                                # in place: H is X, H is R
        a, b = x.clone(), r.clone()
        out, q, s = (a, b)[which], torch.empty_like(Q), torch.empty_like(S)
        G.fp8_add_rmsnorm(a, b, g, 1e-5, out, q, s)
        assert torch.equal(out, H) and torch.equal(q, Q) and torch.equal(s, S)
    q, s = torch.empty_like(Q), torch.empty_like(S)       # no residual: R = -0 adds nothing
    G.fp8_add_rmsnorm(x, None, g, 1e-5, None, q, s)
    G.fp8_add_rmsnorm(x, torch.full_like(x, -0.0), g, 1e-5, None, Q, S)
    assert torch.equal(q, Q) and torch.equal(s, S)


@pytest.mark.parametrize("m,k,ld", [(15001, 200, 201), (4001, 2048, 2049), (1501, 5119, 5119)])
def test_norm_over_many_rounds_of_unaligned_rows(m, k, ld):
    """Rows that 16-byte copies cannot address are loaded when they are due: the same as aligned ones."""
    import post_weight_quantization_18_b200 as G
    X, R, gamma = _norm_case(m, k, "bf16", "bf16", 6)
    x, _ = padded(m, k, torch.bfloat16, ld=ld)
    x.copy_(X)
    y, _ = padded(m, k, torch.bfloat16, ld=-(-k // 8) * 8)
    y.copy_(X)
    r, _ = padded(m, k, torch.bfloat16, ld=-(-k // 8) * 8)
    r.copy_(R)
    outs = []
    for a in (x, y):
        q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
        s = torch.empty((m, -(-k // 128)), device="cuda")
        G.fp8_add_rmsnorm(a, r, gamma.cuda(), 1e-5, None, q, s)
        outs.append((q, s))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    _check_norm(X[-8:], R[-8:], gamma, np.float32(1e-5), None, outs[0][0][-8:], outs[0][1][-8:], "bf16")
