"""GPU parity of fp8_gemm and fp8_gated_gemm with the float64 oracle, and the operators run together.

fp8_gemm's sums are within fp8_util.gemm_bound of the oracle's, then rounded once to Y's type. The
gated pair's h = silu(g) u inherits the bounds of g and u: |silu'| <= 1.1, and exp, the sum, the
quotient and the product are within 8 * 2^-24 of h.
"""
import numpy as np
import pytest
import torch

from fp8_util import DTYPES, HALF_STEP, check_format, codes_of, f64, gemm_bound, padded, untouched
from oracle import fp8 as o

pytestmark = pytest.mark.gpu


def operand(m, k, rows, seed, ld=None, offset=0, scale=1.0):
    """Random e4m3 codes (every finite value) and scales of widely different size, on the GPU: the
    matrix as a view of a buffer whose padding holds e4m3 NaNs, its codes and scales for the oracle."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)).astype(np.float32)
    codes, _ = o.quantize(x, rows)
    S = (scale * np.exp(rng.standard_normal((-(-m // rows), -(-k // 128))))).astype(np.float32)
    view, _ = padded(m, k, torch.uint8, ld=-(-k // 16) * 16 if ld is None else ld, offset=offset)
    view.copy_(torch.from_numpy(codes))
    return view, torch.from_numpy(S).cuda(), codes, S


def check_rounded(Y, ref, bound, dtype):
    """Y is some value within `bound` of ref, rounded to the type. fp16 has no value from 65520 (half
    a step above its largest, 65504) on: round-to-nearest gives an infinity of ref's sign there."""
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    limit = bound + np.maximum((np.abs(ref) + bound) * HALF_STEP[dtype], tiny)
    inf = np.isinf(Y)
    if dtype == "fp16":
        assert np.all(np.abs(ref[inf]) + bound[inf] >= 65520) and np.all(Y[inf] * ref[inf] > 0)
        assert np.all(np.abs(ref[~inf]) - bound[~inf] <= 65520)
    else:
        assert not inf.any()
    err = np.abs(Y[~inf] - ref[~inf])
    assert np.all(err <= limit[~inf]), float(np.max(err / limit[~inf]))


def run_gemm(m, n, k, dtype, seed=0, ldy=None, offy=0, **kw):
    import post_weight_quantization_18_b200 as G
    X, sx, cx, Sx = operand(m, k, 1, seed + 1, **kw)
    W, sw, cw, Sw = operand(n, k, 128, seed + 2, **kw)
    Y, raw = padded(m, n, DTYPES[dtype], ld=n if ldy is None else ldy, offset=offy)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    G.fp8_gemm(X, sx, W, sw, Y, st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0]
    ref, A = o.gemm(cx, Sx, cw, Sw)
    bound = gemm_bound(A, k)
    check_rounded(f64(Y), ref, bound, dtype)
    assert untouched(raw, Y)
    return Y


def run_gated(m, n, k, seed=0, ldq=None, offq=0, scale=0.05, **kw):
    import post_weight_quantization_18_b200 as G
    X, sx, cx, Sx = operand(m, k, 1, seed + 1, scale=scale, **kw)
    Wg, sg, cg, Sg = operand(n, k, 128, seed + 2, scale=scale, **kw)
    Wu, su, cu, Su = operand(n, k, 128, seed + 3, scale=scale, **kw)
    Q, raw_q = padded(m, n, torch.uint8, ld=-(-n // 16) * 16 if ldq is None else ldq, offset=offq)
    S, raw_s = padded(m, -(-n // 128), torch.float32, ld=-(-n // 128) + 1)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    G.fp8_gated_gemm(X, sx, Wg, sg, Wu, su, Q, S, st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0]
    g, Ag = o.gemm(cx, Sx, cg, Sg)
    u, Au = o.gemm(cx, Sx, cu, Su)
    dg, du = gemm_bound(Ag, k), gemm_bound(Au, k)
    h = o.silu(g) * u
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(o.silu(g)) * du + np.abs(h) * 8 * 2.0 ** -24
    check_format(codes_of(Q), S.cpu().numpy(), h, dh)
    assert untouched(raw_q, Q) and untouched(raw_s, S)


SIZES = [
    (1, 128, 128), (1, 1, 1), (1, 4096, 2048), (2, 130, 100), (7, 1000, 1000), (16, 384, 640),
    (17, 256, 1024), (33, 129, 4224), (64, 2304, 1920), (100, 640, 257), (128, 256, 128),
    (129, 257, 129), (200, 2000, 333), (300, 1000, 1000), (515, 1152, 2176), (1030, 2050, 384),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm_matches_oracle(m, n, k, dtype):
    run_gemm(m, n, k, dtype, seed=m + n + k)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_matches_oracle(m, n, k):
    """Gates far from zero: the sigmoid is 0 or 1 nearly everywhere."""
    run_gated(m, n, k, seed=m + n + k)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_matches_oracle_where_the_sigmoid_bends(m, n, k):
    run_gated(m, n, k, seed=m + n + k, scale=0.05 / (64.0 * k ** 0.25))


# Shapes that take each variant of the kernels on a B200: clusters of different size along K, tiles of
# 32, 64, 96 (which span two weight blocks) and 128 weight rows, several rounds of CTAs, output rows that
# 16-byte stores cannot address, pairs of CTAs with odd numbers of row tiles.
VARIANTS = [
    (8, 4224, 4096), (32, 11008, 512), (31, 129, 8200), (16, 20000, 384),
    (40, 512, 4096), (40, 480, 5200), (33, 8192, 256), (100, 11008, 256), (40, 14000, 200),
    (150, 8192, 256), (150, 8191, 264), (40, 11003, 256), (34, 2999, 1024), (130, 4097, 300),
    (1030, 2051, 264), (700, 9000, 136), (2100, 1100, 512),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", VARIANTS)
def test_gemm_variants(m, n, k, dtype):
    run_gemm(m, n, k, dtype, seed=m + n + k)


# The gated pair's own: its largest tile with the weight as the MMAs' M, and the smallest without.
GATED_VARIANTS = [
    (40, 6144, 256), (129, 3000, 1536), (64, 4224, 4096), (64, 20000, 384), (50, 129, 8200),
    (33, 1, 1), (65, 512, 4096), (72, 1000, 1100), (66, 2304, 2048), (80, 6144, 256),
    (90, 13999, 256),
]


@pytest.mark.parametrize("m,n,k", VARIANTS + GATED_VARIANTS)
def test_gated_variants(m, n, k):
    run_gated(m, n, k, seed=m + n + k, scale=0.05 / (64.0 * k ** 0.25))


@pytest.mark.parametrize("m", [3, 40, 140])
@pytest.mark.parametrize("kw", [dict(ld=300), dict(ld=301), dict(ld=304, offset=1),
                                dict(ld=320, offset=8), dict(ld=384, offset=16)])
def test_operands_of_any_alignment(m, kw):
    """Pitches and bases that are not multiples of 16 bytes, and some that are."""
    run_gemm(m, 260, 300, "bf16", seed=m, **kw)
    run_gated(m, 260, 300, seed=m, **kw)


@pytest.mark.parametrize("m", [3, 140])
@pytest.mark.parametrize("dtype,ldy", [("bf16", 261), ("fp16", 264), ("fp32", 263), ("fp32", 268)])
def test_output_pitches(m, dtype, ldy):
    run_gemm(m, 260, 512, dtype, seed=m, ldy=ldy)
    run_gated(m, 260, 512, seed=m, ldq=ldy, offq=ldy % 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offy", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("m,n,ldy", [(40, 1, 1), (40, 2, 3), (41, 3, 3), (130, 15, 17), (40, 17, 17),
                                     (70, 33, 34), (129, 127, 131), (300, 129, 129), (40, 130, 132),
                                     (1030, 4099, 4099), (1025, 4130, 4134)])
def test_output_views_of_any_alignment(m, n, ldy, offy, dtype):
    """Rows that begin at any multiple of the element's size, and end inside a store."""
    run_gemm(m, n, 136, dtype, seed=m + n, ldy=ldy, offy=offy)


def test_scale_pitches_and_stacked_weights():
    """Scales as columns of wider arrays; gate and up as the halves of one stacked weight."""
    import post_weight_quantization_18_b200 as G
    m, n, k = 70, 384, 512
    X, sx, cx, Sx = operand(m, k, 1, 1, scale=0.05)
    W, sw, cw, Sw = operand(2 * n, k, 128, 2, scale=0.05)
    wide_x = torch.full((m, 9), float("nan"), device="cuda")
    wide_x[:, 2:6] = sx
    wide_w = torch.full((2 * n // 128, 7), float("nan"), device="cuda")
    wide_w[:, 3:] = sw
    out = G.fp8.empty(m, n)
    G.fp8_gated_gemm(X, wide_x[:, 2:6], W[:n], wide_w[:3, 3:], W[n:], wide_w[3:, 3:], out.q,
                     out.scales)
    want = G.fp8.empty(m, n)
    G.fp8_gated_gemm(X, sx, W[:n].clone(), sw[:3].clone(), W[n:].clone(), sw[3:].clone(), want.q,
                     want.scales)
    assert torch.equal(out.q.view(torch.uint8), want.q.view(torch.uint8))
    assert torch.equal(out.scales, want.scales)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_nan_stays_in_its_row_or_column(m):
    """A NaN scale of a row, or of a weight block, reaches that row, or those columns, alone."""
    import post_weight_quantization_18_b200 as G
    n, k = 400, 640
    X, sx, _, _ = operand(m, k, 1, 5)
    W, sw, _, _ = operand(n, k, 128, 6)
    Y0 = torch.empty((m, n), device="cuda")
    G.fp8_gemm(X, sx, W, sw, Y0)
    assert not torch.isnan(Y0).any()
    sw2, sx2, W2 = sw.clone(), sx.clone(), W.clone()
    sw2[1, 3] = float("nan")
    sx2[m // 2, 4] = float("nan")
    W2[300, 639] = 0x7F
    Y = torch.empty((m, n), device="cuda")
    G.fp8_gemm(X, sx2, W2, sw2, Y)
    want = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    want[:, 128:256] = True
    want[m // 2] = True
    want[:, 300] = True
    assert torch.equal(torch.isnan(Y), want)
    assert torch.equal(Y[~want], Y0[~want])


@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (40, 512, 4096), (300, 640, 1024),
                                   (1030, 2050, 384)])
def test_status_repeats_and_capture(m, n, k):
    """Skipped while the status holds an error; two calls give the same bits, and so does a replay
    of a captured pair, beside a direct call on another stream."""
    import post_weight_quantization_18_b200 as G
    X, sx, _, _ = operand(m, k, 1, 7, scale=0.1)
    W, sw, _, _ = operand(n, k, 128, 8, scale=0.1)
    W2, sw2, _, _ = operand(n, k, 128, 9, scale=0.1)
    bad = torch.tensor([16, 0], dtype=torch.int32, device="cuda")
    Y = torch.full((m, n), 3.0, device="cuda")
    out = G.fp8.empty(m, n)
    out.q.view(torch.uint8).fill_(9)
    out.scales.fill_(5.0)
    G.fp8_gemm(X, sx, W, sw, Y, bad)
    G.fp8_gated_gemm(X, sx, W, sw, W2, sw2, out.q, out.scales, bad)
    assert (Y == 3.0).all() and (out.q.view(torch.uint8) == 9).all() and (out.scales == 5.0).all()
    G.fp8_gemm(X, sx, W, sw, Y)
    G.fp8_gated_gemm(X, sx, W, sw, W2, sw2, out.q, out.scales)
    Yg, outg = torch.zeros_like(Y), G.fp8.empty(m, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.fp8_gemm(X, sx, W, sw, Yg)
        G.fp8_gated_gemm(X, sx, W, sw, W2, sw2, outg.q, outg.scales)
    side = torch.cuda.Stream()
    Ys = torch.zeros_like(Y)
    for _ in range(3):
        Yg.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            G.fp8_gemm(X, sx, W, sw, Ys)
        torch.cuda.synchronize()
        assert torch.equal(Y, Yg) and torch.equal(Y, Ys)
        assert torch.equal(out.q.view(torch.uint8), outg.q.view(torch.uint8))
        assert torch.equal(out.scales, outg.scales)


@pytest.mark.parametrize("m", [0, 1, 5, 150])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_mlp_block(m, dtype):
    """norm -> gated pair -> down projection -> next norm, as a decoder block runs them, against the
    composition in float64 of each operator on the codes the one before it gave."""
    import post_weight_quantization_18_b200 as G
    d, f = 640, 1100
    g = torch.Generator().manual_seed(m)
    rnd = lambda *s: torch.randn(s, generator=g)
    X, R = rnd(m, d).to(DTYPES[dtype]).cuda(), (2 * rnd(m, d)).to(DTYPES[dtype]).cuda()
    gamma = (1 + 0.1 * rnd(d)).cuda()
    Ws = [(0.05 * rnd(f, d)).cuda(), (0.05 * rnd(f, d)).cuda(), (0.05 * rnd(d, f)).cuda()]
    mlp = G.fp8.GatedMLP.from_weights(gamma, *Ws)
    y, h = mlp(X, R)
    q2, h2 = G.fp8.add_rmsnorm(y, h, gamma)
    torch.cuda.synchronize()
    assert y.dtype == DTYPES[dtype] and y.shape == (m, d) and h2.shape == (m, d)
    if m == 0:
        return
    xq, hh = G.fp8.add_rmsnorm(X, R, gamma)
    hid = G.fp8.gated(xq, mlp.gate, mlp.up)
    assert torch.equal(hh, h) and torch.equal(G.fp8.linear(hid, mlp.down, X.dtype), y)
    # the whole block against 64 bits without any 8-bit rounding: what the format costs, 2^-4 half
    # steps of weights and activations that average out over the sums
    hn, yn = o.add_rmsnorm(f64(X), f64(R), f64(gamma), 1e-5)
    gg, uu = yn @ f64(Ws[0]).T, yn @ f64(Ws[1]).T
    ref = (o.silu(gg) * uu) @ f64(Ws[2]).T
    rel = np.linalg.norm(f64(y) - ref) / np.linalg.norm(ref)
    assert rel <= 0.15, rel
    # and exactly, operator by operator, on the codes
    ref, A = o.gemm(codes_of(hid.q), hid.scales.cpu().numpy(), codes_of(mlp.down.q),
                    mlp.down.scales.cpu().numpy())
    b = gemm_bound(A, f)
    assert np.all(np.abs(f64(y) - ref) <= b + (np.abs(ref) + b) * HALF_STEP[dtype] + 2.0 ** -25)
    _, yn = o.add_rmsnorm(f64(y), f64(h), f64(gamma), np.float32(1e-5))
    check_format(codes_of(q2.q), q2.scales.cpu().numpy(), yn, np.abs(yn) * 2.0 ** -19)


def test_linear_on_quantized_layer_has_the_formats_error():
    """quantize_weight / quantize_activations / linear on a layer's own tensors."""
    import post_weight_quantization_18_b200 as G
    m, n, k = 50, 384, 1000
    X = torch.randn((m, k), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    W = (0.02 * torch.randn((n, k), generator=torch.Generator().manual_seed(2))).bfloat16().cuda()
    x, w = G.fp8.quantize_activations(X), G.fp8.quantize_weight(W)
    Y = G.fp8.linear(x, w, torch.float32)
    ref, A = o.gemm(codes_of(x.q), x.scales.cpu().numpy(), codes_of(w.q), w.scales.cpu().numpy())
    assert np.all(np.abs(f64(Y) - ref) <= gemm_bound(A, k) + np.abs(ref) * 2.0 ** -24)
    np.testing.assert_allclose(f64(x.dequantize()) @ f64(w.dequantize()).T, ref, rtol=0,
                               atol=float(A.max()) * 2.0 ** -22)


def test_binding_refuses_wrong_operands():
    import post_weight_quantization_18_b200 as G
    q = torch.zeros((4, 256), dtype=torch.uint8, device="cuda")
    s, sw = torch.zeros((4, 2), device="cuda"), torch.zeros((1, 2), device="cuda")
    Y = torch.zeros((4, 4), device="cuda")
    with pytest.raises(ValueError, match="float8_e4m3fn or uint8"):
        G.fp8_gemm(q.to(torch.int32), s, q, sw, Y)
    with pytest.raises(ValueError, match=r"sw must be \[1, 2\]"):
        G.fp8_gemm(q, s, q, s, Y)
    with pytest.raises(ValueError, match="torch.float32"):
        G.fp8_gemm(q, s.half(), q, sw, Y)
    with pytest.raises(ValueError, match=r"W must be \[4, 256\]"):
        G.fp8_gemm(q, s, q[:, :128], sw, Y)
    with pytest.raises(ValueError, match=r"Y must be \[4, 4\]"):
        G.fp8_gemm(q, s, q, sw, Y[:3])
    with pytest.raises(ValueError, match="CUDA"):
        G.fp8_gemm(q, s, q.cpu(), sw, Y)
    with pytest.raises(ValueError, match="dev_status"):
        G.fp8_gemm(q, s, q, sw, Y, torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="unit stride"):
        G.fp8_gemm(q, s, q, sw, torch.zeros((4, 4), device="cuda").t())
    with pytest.raises(ValueError, match=r"Q must be \[4, 4\]"):
        G.fp8_gated_gemm(q, s, q, sw, q, sw, q, s)


# Gates around the points where exp(-g) passes 2^126 (-87.34), 2^128 (-88.72) and, as exp(g), the smallest
# subnormal number (-103.97), around -64 and 0.
GATES = [-150.0, -120.0, -104.5, -103.9, -100.0, -95.0, -89.0, -88.75, -88.7, -88.5, -88.0, -87.5, -87.375,
         -87.25, -87.0, -80.0, -64.5, -64.0, -63.5, -40.0, -1.0, -0.5, 0.25, 3.0, 30.0, 87.0, 88.0, 89.0]


@pytest.mark.parametrize("m,n,ld", [
    (10, 200, 16), (28, 130, 16), (60, 4864, 16),         # few rows: 16, 32, 64 of them a tile
    (100, 300, 16), (100, 6144, 16), (100, 11008, 16),    # tiles of 32, 64 and 128 weight rows
    (300, 4096, 16), (40, 130, 17),                       # pairs of CTAs; operands TMA cannot address
])
def test_gate_far_below_zero(m, n, ld):
    """silu(g) u with g of -150 to 89, exact in the sums, and u so large that h is an ordinary number: one
    column of K, x = 1 with the scale |g|, Wg = -1 or 1, and Wu = the e4m3 numbers with the scale 2^100.
    The sigmoid e / (1 + e), e = exp(g), is off by 9 * 2^-24 of itself (exp 2 ulp, of 2^-23 at most: 4; the sum
    1, the quotient of 2 ulp 4) and, being a subnormal number from -87.3 on, by 2 ulp of exp and 1 of the
    quotient, 2^-149 each: 2^-147 at most. Two products and u itself: 3 * 2^-24."""
    import post_weight_quantization_18_b200 as G
    gates = np.resize(np.array(GATES, np.float32), m)
    for sign in (-1, 1):
        rows = np.where(np.sign(gates) == sign, gates, np.float32(sign))
        buf = lambda r: padded(r, 1, torch.uint8, ld=ld)[0]
        X, Wg, Wu = buf(m), buf(n), buf(n)
        X.fill_(0x38)                                     # 1
        Wg.fill_(0x38 if sign > 0 else 0xB8)
        codes = np.resize(np.arange(1, 127, dtype=np.uint8), n)
        codes[1::2] |= 0x80
        Wu.copy_(torch.from_numpy(codes)[:, None])
        sx = torch.from_numpy(np.abs(rows))[:, None].cuda()
        sg = torch.ones((-(-n // 128), 1), device="cuda")
        out = G.fp8.empty(m, n)
        G.fp8_gated_gemm(X, sx, Wg, sg, Wu, sg * 2.0 ** 100, out.q, out.scales)
        g = rows.astype(np.float64)[:, None]
        u = np.abs(g) * o.decode(codes)[None] * 2.0 ** 100
        h = g * u / (1 + np.exp(-g))
        dh = np.abs(h) * 12 * 2.0 ** -24 + np.abs(g * u) * 2.0 ** -147
        check_format(codes_of(out.q), out.scales.cpu().numpy(), h, dh)
