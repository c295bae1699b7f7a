"""The 8-bit floating point operators as calls to measure: the blocks of 128 that carry one scale,
the norm that feeds them, the matrix product that reads them and the gated pair of products.

Format. A matrix in 8 bits holds e4m3 numbers and fp32 scales. Activations [m, k] have one scale
for each row and 128 consecutive columns (scales [m, ceil(k / 128)]); weights [n, k] have one for
each block of 128 rows and 128 columns (scales [ceil(n / 128), ceil(k / 128)]). The value of an
element is its e4m3 number times its block's scale, and a block's scale is the largest magnitude
in it divided by 448 (1 for a block of zeros). Rows are stored with a pitch that is a multiple of
16 bytes, as the framework's own allocations are.

Operators (case["op"]):
  quantize   [m, k] in 16 or 32 bits -> e4m3 and scales, blocks of 1 or 128 rows
  norm       h = x + r; e4m3 and scales of h / sqrt(mean(h^2) + eps) * gamma; h itself
  gemm       Y = X W^T of two matrices in this format
  gated      e4m3 and scales of silu(X Wg^T) * (X Wu^T)
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 1e-5
_E4M3_MAX = 448.0


def listed():
    return [
        # activations of one decoding step of 16 sequences on their way into an attention
        # projection (4096 wide)
        {"name": "quantize_rows_16x4096", "op": "quantize", "m": 16, "k": 4096, "rows": 1, "type": "bf16"},
        # activations of a prompt chunk before a down projection of 11008 columns
        {"name": "quantize_rows_4096x11008", "op": "quantize", "m": 4096, "k": 11008, "rows": 1, "type": "fp16"},
        # the largest weight there is here, 8192 x 28672, brought into the format once at load
        {"name": "quantize_weight_8192x28672", "op": "quantize", "m": 8192, "k": 28672, "rows": 128, "type": "bf16"},
        # one token of each of 4 sequences between two blocks of a 4096-wide model
        {"name": "norm_4x4096", "op": "norm", "m": 4, "k": 4096, "type": "bf16"},
        # a prompt of 8192 tokens, 5120 wide
        {"name": "norm_8192x5120", "op": "norm", "m": 8192, "k": 5120, "type": "bf16"},
        # an odd batch, a width that is no multiple of 128, a residual stream kept in fp32
        {"name": "norm_333x1000_fp32", "op": "norm", "m": 333, "k": 1000, "type": "fp32"},
        # one token through a 4096 x 4096 projection: latency
        {"name": "gemm_1x4096x4096", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "type": "bf16"},
        # 32 sequences decoding, through a 11008 x 4096 projection: the weight's bytes
        {"name": "gemm_32x11008x4096", "op": "gemm", "m": 32, "n": 11008, "k": 4096, "type": "bf16"},
        # a ragged prompt, widths that are no multiples of 128, fp32 out
        {"name": "gemm_300x1000x1000_fp32", "op": "gemm", "m": 300, "n": 1000, "k": 1000, "type": "fp32"},
        # a long prompt through the 8192 x 28672 down projection: the tensor cores' rate
        {"name": "gemm_8192x8192x28672", "op": "gemm", "m": 8192, "n": 8192, "k": 28672, "type": "bf16"},
        # 8 sequences decoding through gate and up projections of 11008 x 4096
        {"name": "gated_8x11008x4096", "op": "gated", "m": 8, "n": 11008, "k": 4096},
        # a prompt of 2000 tokens (not a multiple of 128) through 13824 x 5120
        {"name": "gated_2000x13824x5120", "op": "gated", "m": 2000, "n": 13824, "k": 5120},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A model's width: mostly a multiple of 128, at times a multiple of 8 or any number."""
    v, kind = _log_int(rng, lo, hi), rng.random()
    return max(128, v // 128 * 128) if kind < 0.6 else max(8, v // 8 * 8) if kind < 0.8 else v


def draw(rng):
    op = rng.choice(["quantize", "norm", "gemm", "gemm", "gated"])
    if op == "quantize":
        rows = rng.choice([1, 128])
        k = _width(rng, 128, 28672)
        return {"op": op, "m": _log_int(rng, 1, min(16384, 100_000_000 // k)), "k": k, "rows": rows,
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "norm":
        k = _width(rng, 128, 16384)
        return {"op": op, "m": _log_int(rng, 1, min(16384, 100_000_000 // k)), "k": k,
                "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    n, k = _width(rng, 128, 14336), _width(rng, 128, 14336)
    m = _log_int(rng, 1, min(8192, max(2, 200_000_000_000 // (n * k))))
    if op == "gemm":
        return {"op": op, "m": m, "n": n, "k": k, "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    return {"op": op, "m": m, "n": n, "k": k}


def _groups(n):
    return -(-n // 128)


def _fp8_buffer(m, k):
    """[m, k] of e4m3 whose rows are a multiple of 16 bytes apart."""
    return torch.zeros((m, -(-k // 16) * 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :k]


def _scales_buffer(m, k, rows):
    return torch.zeros((-(-m // rows), _groups(k)), dtype=torch.float32, device="cuda")


def _activations(gen, m, k):
    """Normal values with channels of very different size, a few of them large."""
    channel = torch.exp(0.7 * torch.randn(k, generator=gen, device="cuda"))
    channel[torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 1000)]] *= 20.0
    return torch.randn((m, k), generator=gen, device="cuda") * channel


def _blocks(x, rows):
    """x [m, k] padded with zeros and seen as [row blocks, rows, column blocks, 128]."""
    m, k = x.shape
    mp, kp = -(-m // rows) * rows, _groups(k) * 128
    if (mp, kp) != (m, k):
        padded = x.new_zeros((mp, kp))
        padded[:m, :k] = x
        x = padded
    return x.view(mp // rows, rows, kp // 128, 128)


def _quantize(x, rows):
    """The plain form: (e4m3 [m, k], scales) of x in fp32."""
    m, k = x.shape
    b = _blocks(x, rows)
    scale = b.abs().amax(dim=(1, 3)) / _E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale.clamp(min=2.0 ** -126))
    q = (b * (1.0 / scale)[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(b.shape[0] * rows, -1)[:m, :k], scale


def _dequantize(q, scales, rows):
    """The fp32 values of a matrix in the format."""
    m, k = q.shape
    b = _blocks(q.to(torch.float32), rows)
    return (b * scales[:, None, :, None]).view(b.shape[0] * rows, -1)[:m, :k]


def _held(x, rows):
    """x as a program holds it: in the format, rows a multiple of 16 bytes apart."""
    q, s = _quantize(x, rows)
    buf = _fp8_buffer(*x.shape)
    buf.copy_(q)
    return buf, s.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    st = {"op": op}
    if op == "quantize":
        rows, t = case["rows"], _TYPES[case["type"]]
        x = _activations(gen, m, k) if rows == 1 else 0.015 * torch.randn((m, k), generator=gen, device="cuda")
        st.update(x=x.to(t), rows=rows, q=_fp8_buffer(m, k), s=_scales_buffer(m, k, rows))
    elif op == "norm":
        t = _TYPES[case["type"]]
        st.update(x=torch.randn((m, k), generator=gen, device="cuda").to(t),
                  r=_activations(gen, m, k).to(t),
                  gamma=(1.0 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(t),
                  h=torch.zeros((m, k), dtype=t, device="cuda"),
                  q=_fp8_buffer(m, k), s=_scales_buffer(m, k, 1))
    else:
        n = case["n"]
        st["x"], st["sx"] = _held(_activations(gen, m, k), 1)
        if op == "gemm":
            st["w"], st["sw"] = _held(0.02 * torch.randn((n, k), generator=gen, device="cuda"), 128)
            st["y"] = torch.zeros((m, n), dtype=_TYPES[case["type"]], device="cuda")
        else:
            st["wg"], st["sg"] = _held(0.02 * torch.randn((n, k), generator=gen, device="cuda"), 128)
            st["wu"], st["su"] = _held(0.02 * torch.randn((n, k), generator=gen, device="cuda"), 128)
            st.update(q=_fp8_buffer(m, n), s=_scales_buffer(m, n, 1))
    return st


def _run_own(st):
    import post_weight_quantization_18_b200 as G
    op = st["op"]
    if op == "quantize":
        G.fp8_quantize(st["x"], st["q"], st["s"], st["rows"])
        return st["q"], st["s"]
    if op == "norm":
        G.fp8_add_rmsnorm(st["x"], st["r"], st["gamma"], _EPS, st["h"], st["q"], st["s"])
        return st["q"], st["s"], st["h"]
    if op == "gemm":
        G.fp8_gemm(st["x"], st["sx"], st["w"], st["sw"], st["y"])
        return st["y"]
    G.fp8_gated_gemm(st["x"], st["sx"], st["wg"], st["sg"], st["wu"], st["su"], st["q"], st["s"])
    return st["q"], st["s"]


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "quantize":
        return _quantize(st["x"].to(torch.float32), st["rows"])
    if op == "norm":
        h = st["x"].to(torch.float32) + st["r"].to(torch.float32)
        y = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + _EPS) * st["gamma"].to(torch.float32)
        q, s = _quantize(y, 1)
        return q, s, h.to(st["h"].dtype)
    x = _dequantize(st["x"], st["sx"], 1)
    if op == "gemm":
        return torch.matmul(x, _dequantize(st["w"], st["sw"], 128).t()).to(st["y"].dtype)
    g = torch.matmul(x, _dequantize(st["wg"], st["sg"], 128).t())
    u = torch.matmul(x, _dequantize(st["wu"], st["su"], 128).t())
    return _quantize(g / (1.0 + torch.exp(-g)) * u, 1)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    gk = _groups(k)
    if op == "quantize":  # x once, its e4m3 numbers and scales once; |x| and its maximum, the product
        return {"bytes": m * k * (_BYTES[case["type"]] + 1) + 4 * gk * -(-m // case["rows"]), "flops": 3 * m * k}
    if op == "norm":  # x, r and gamma once, h, the e4m3 numbers and scales once
        b = _BYTES[case["type"]]
        return {"bytes": m * k * (3 * b + 1) + k * b + 4 * m * gk, "flops": 8 * m * k}
    n = case["n"]
    gn = _groups(n)
    held = m * k + 4 * m * gk
    if op == "gemm":
        return {"bytes": held + n * k + 4 * gn * gk + m * n * _BYTES[case["type"]], "flops": 2 * m * n * k}
    return {"bytes": held + 2 * (n * k + 4 * gn * gk) + m * n + 4 * m * gn, "flops": 4 * m * n * k + 6 * m * n}


def _scale_of_column(scales, rows, m, k):
    """The scale of every element, as a [m, k] matrix of 64 bits."""
    i = torch.arange(m, device=scales.device) // rows
    j = torch.arange(k, device=scales.device) // 128
    return scales.double()[i][:, j]


def _exact_format(y, rows):
    """From 64-bit values: the numbers before their rounding to e4m3, and the scales."""
    m, k = y.shape
    top = torch.zeros((-(-m // rows), _groups(k)), dtype=torch.float64, device=y.device)
    i = (torch.arange(m, device=y.device) // rows)[:, None].expand(m, _groups(k))
    per_row = torch.stack([c.abs().amax(dim=1) for c in y.split(128, dim=1)], dim=1)
    top.scatter_reduce_(0, i, per_row, "amax")
    scales = torch.where(top > 0, (top / _E4M3_MAX).clamp(min=2.0 ** -126), torch.ones_like(top))
    return y / _scale_of_column(scales, rows, m, k), scales


def exact(case, seed):
    st = prepare(case, seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        return _exact_format(st["x"].double(), st["rows"])
    if op == "norm":
        h = st["x"].double() + st["r"].double()
        rms = torch.linalg.vector_norm(h, dim=1, keepdim=True) / math.sqrt(k)
        q, s = _exact_format(h * st["gamma"].double() / torch.sqrt(rms * rms + _EPS), 1)
        return q, s, h
    x = st["x"].double() * _scale_of_column(st["sx"], 1, m, k)
    if op == "gemm":
        return x @ (st["w"].double() * _scale_of_column(st["sw"], 128, case["n"], k)).T
    g = x @ (st["wg"].double() * _scale_of_column(st["sg"], 128, case["n"], k)).T
    u = x @ (st["wu"].double() * _scale_of_column(st["su"], 128, case["n"], k)).T
    return _exact_format(g * torch.sigmoid(g) * u, 1)
