"""The e4m3 operators as a program runs them: one after the other with other kernels between, on several
streams, captured, with operands and outputs of more than 2^32 bytes. A kernel of theirs may start
before the kernel ahead of it in the stream has ended; what it reads and writes must not show it."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from fp8_util import check_format, codes_of, f64, gemm_bound
from oracle import fp8 as o

pytestmark = pytest.mark.gpu


def _weights(n, k, seed, count=1):
    import post_weight_quantization_18_b200 as G
    g = torch.Generator().manual_seed(seed)
    return [G.fp8.quantize_weight((torch.randn((n, k), generator=g) / k ** 0.5).cuda())
            for _ in range(count)]


@pytest.mark.parametrize("m", [1, 7, 40, 300])
def test_chain_with_other_kernels_between(m):
    """Each call's input is written by the kernel just before it and overwritten by the one just after:
    50 rounds in a row, without waiting, give what one call at a time gives."""
    import post_weight_quantization_18_b200 as G
    d, f = 1024, 1536
    wg, wu = _weights(f, d, 1, 2)
    wd, = _weights(d, f, 2)
    gamma = torch.ones(d, device="cuda")
    g = torch.Generator().manual_seed(m)
    start = torch.randn((m, d), generator=g).bfloat16().cuda()

    def step(x, r, y, h, xq, hq, wait):
        s = (lambda: torch.cuda.synchronize()) if wait else (lambda: None)
        G.fp8_add_rmsnorm(x, r, gamma, 1e-5, h, xq.q, xq.scales); s()
        x.fill_(float("nan")); s()
        G.fp8_gated_gemm(xq.q, xq.scales, wg.q, wg.scales, wu.q, wu.scales, hq.q, hq.scales); s()
        xq.scales.fill_(float("nan")); s()
        G.fp8_gemm(hq.q, hq.scales, wd.q, wd.scales, y); s()
        hq.scales.fill_(float("nan")); s()
        r.copy_(h); s()
        torch.mul(y, 0.5, out=x); s()

    def run(wait):
        x, r = start.clone(), (2 * start).clone()
        y, h = torch.zeros_like(x), torch.zeros_like(x)
        xq, hq = G.fp8.empty(m, d), G.fp8.empty(m, f)
        for _ in range(50):
            step(x, r, y, h, xq, hq, wait)
        torch.cuda.synchronize()
        return x, r
    a, b = run(False), run(True)
    assert torch.isfinite(a[0]).all() and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_hand_over_and_run_side_by_side():
    """A producer's and a consumer's stream with events between them, while a third stream runs the
    large kernels; every result as if alone."""
    import post_weight_quantization_18_b200 as G
    w, = _weights(2048, 1024, 3)
    big_w, = _weights(4096, 2048, 4)
    g = torch.Generator().manual_seed(5)
    X = [torch.randn((6, 1024), generator=g).bfloat16().cuda() for _ in range(30)]
    B = G.fp8.quantize_activations(torch.randn((700, 2048), generator=g).cuda())
    want = [G.fp8.linear(G.fp8.quantize_activations(x), w) for x in X]
    want_big = G.fp8.linear(B, big_w)
    torch.cuda.synchronize()
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
    got, bigs = [], []
    q = [G.fp8.empty(6, 1024) for _ in range(2)]
    freed = [torch.cuda.Event() for _ in range(2)]
    ys = [torch.empty_like(want[0]) for _ in X]
    yb = [torch.empty_like(want_big) for _ in range(10)]
    torch.cuda.synchronize()
    for i, x in enumerate(X):
        with torch.cuda.stream(s1):
            if i >= 2:
                s1.wait_event(freed[i % 2])
            G.fp8_quantize(x, q[i % 2].q, q[i % 2].scales)
            done = torch.cuda.Event()
            done.record(s1)
        with torch.cuda.stream(s2):
            s2.wait_event(done)
            G.fp8_gemm(q[i % 2].q, q[i % 2].scales, w.q, w.scales, ys[i])
            freed[i % 2] = torch.cuda.Event()
            freed[i % 2].record(s2)
        if i % 3 == 0:
            with torch.cuda.stream(s3):
                G.fp8_gemm(B.q, B.scales, big_w.q, big_w.scales, yb[i // 3])
    torch.cuda.synchronize()
    for y, t in zip(ys, want):
        assert torch.equal(y, t)
    for y in yb:
        assert torch.equal(y, want_big)


def test_two_graphs_of_the_same_operators():
    """Two graphs captured over different buffers replay at once, on two streams, and interleaved on one:
    nothing is shared between calls."""
    import post_weight_quantization_18_b200 as G
    wg, wu = _weights(1024, 768, 6, 2)
    gamma = torch.ones(768, device="cuda")
    g = torch.Generator().manual_seed(7)
    bufs = []
    for m in (5, 64):
        x = torch.randn((m, 768), generator=g).bfloat16().cuda()
        bufs.append((x, torch.zeros_like(x), G.fp8.empty(m, 768), G.fp8.empty(m, 1024)))

    def body(b):
        x, h, xq, hq = b
        G.fp8_add_rmsnorm(x, x, gamma, 1e-5, h, xq.q, xq.scales)
        G.fp8_gated_gemm(xq.q, xq.scales, wg.q, wg.scales, wu.q, wu.scales, hq.q, hq.scales)
    graphs, want = [], []
    for b in bufs:
        body(b)
        torch.cuda.synchronize()
        want.append((b[3].q.view(torch.uint8).clone(), b[3].scales.clone()))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            body(b)
        graphs.append(gr)
    s = [torch.cuda.Stream() for _ in range(2)]
    for rounds in range(20):
        for b in bufs:
            b[3].scales.zero_()
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(s[i if rounds % 2 else 0]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for b, (q, sc) in zip(bufs, want):
            assert torch.equal(b[3].q.view(torch.uint8), q) and torch.equal(b[3].scales, sc)


def test_first_calls_may_be_captured():
    """A process whose first calls are recorded: nothing that the calls set up once breaks the capture."""
    code = """
import torch, post_weight_quantization_18_b200 as G
X = torch.randn(40, 512, device="cuda").bfloat16()
W = torch.randn(640, 512, device="cuda").bfloat16()
x, w, y = G.fp8.empty(40, 512), G.fp8.empty(640, 512, 128), torch.zeros(40, 640, device="cuda")
z = torch.zeros(3, 640, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    G.fp8_quantize(X, x.q, x.scales)
    G.fp8_quantize(W, w.q, w.scales, 128)
    G.fp8_gemm(x.q, x.scales, w.q, w.scales, y)
    G.fp8_gemm(x.q[:3], x.scales[:3], w.q, w.scales, z)
g.replay()
torch.cuda.synchronize()
ref = x.dequantize() @ w.dequantize().T
assert (y - ref).abs().max() < 1e-2 * ref.abs().max(), "product"
assert (z - ref[:3]).abs().max() < 1e-2 * ref.abs().max(), "few rows"
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_operand_past_32_bits():
    """X of 4.9 GB: the last rows come out as they do alone."""
    import post_weight_quantization_18_b200 as G
    m, n, k = 300_000, 256, 16_384
    w, = _weights(n, k, 8)
    x = G.fp8.empty(m, k)
    x.q.view(torch.uint8).zero_()
    x.scales.fill_(1.0)
    tail = G.fp8.quantize_activations(
        torch.randn((300, k), generator=torch.Generator().manual_seed(9)).cuda())
    x.q[-300:] = tail.q
    x.scales[-300:] = tail.scales
    Y = G.fp8.linear(x, w)
    alone = G.fp8.linear(tail, w)
    ref, A = o.gemm(codes_of(tail.q), tail.scales.cpu().numpy(), codes_of(w.q), w.scales.cpu().numpy())
    b = gemm_bound(A, k)
    for y in (Y[-300:], alone):
        assert np.all(np.abs(f64(y) - ref) <= b + (np.abs(ref) + b) * 2.0 ** -8)
    assert not Y[:-300].any()


def test_output_past_32_bits():
    """Y of 2.5e9 elements, and the gated pair's output of 4.9 GB's worth of rows at its end."""
    import post_weight_quantization_18_b200 as G
    m, n, k = 300_000, 8_192, 128
    g = torch.Generator().manual_seed(10)
    w, w2 = _weights(n, k, 11, 2)
    x = G.fp8.empty(m, k)
    x.q.view(torch.uint8).zero_()
    x.scales.fill_(1.0)
    tail = G.fp8.quantize_activations(torch.randn((130, k), generator=g).cuda())
    x.q[-130:] = tail.q
    x.scales[-130:] = tail.scales
    Y = G.fp8.linear(x, w)
    ref, A = o.gemm(codes_of(tail.q), tail.scales.cpu().numpy(), codes_of(w.q), w.scales.cpu().numpy())
    b = gemm_bound(A, k)
    assert np.all(np.abs(f64(Y[-130:]) - ref) <= b + (np.abs(ref) + b) * 2.0 ** -8)
    assert not Y[:-130].any()
    del Y
    out = G.fp8.gated(x, w, w2)
    u, Au = o.gemm(codes_of(tail.q), tail.scales.cpu().numpy(), codes_of(w2.q), w2.scales.cpu().numpy())
    h = o.silu(ref) * u
    dg, du = b, gemm_bound(Au, k)
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(o.silu(ref)) * du + np.abs(h) * 8 * 2.0 ** -24
    check_format(codes_of(out.q[-130:]), out.scales[-130:].cpu().numpy(), h, dh)
    assert not (out.q[:-130].view(torch.uint8) & 0x7F).any() and (out.scales[:-130] == 1).all()


def test_a_failed_launch_does_not_fail_the_next_call():
    """A call on a stream whose capture has been invalidated is refused by the runtime; the error is that
    call's alone, and the library's next one, whose launch is fine, says so."""
    code = """
import ctypes, torch, post_weight_quantization_18_b200 as G
X = torch.randn(40, 512, device="cuda").bfloat16()
x = G.fp8.empty(40, 512)
s = torch.cuda.Stream()
torch.cuda.synchronize()
rt = ctypes.CDLL("libcudart.so.12")
raw, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
assert rt.cudaStreamBeginCapture(raw, 1) == 0
assert rt.cudaStreamSynchronize(raw) != 0
with torch.cuda.stream(s):
    try:
        G.fp8_quantize(X, x.q, x.scales)
        print("not refused")
    except G.GPTQError as e:
        assert e.code == 4, e.code
assert rt.cudaStreamEndCapture(raw, ctypes.byref(graph)) != 0
rt.cudaGetLastError()
W = torch.randn(8, 256, device="cuda")
try:
    G.rtn(W)
except G.GPTQError as e:
    print("failed by the call before:", e)
torch.cuda.synchronize()
G.fp8_quantize(X, x.q, x.scales)
torch.cuda.synchronize()
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_modules_example_runs():
    """The lines at the top of fp8.py, as they stand there."""
    import post_weight_quantization_18_b200 as G
    lines = [l[4:] for l in G.fp8.__doc__.splitlines() if l.startswith("    ")]
    assert len(lines) >= 4
    rnd = lambda *s: torch.randn(s, generator=torch.Generator().manual_seed(len(s))).bfloat16().cuda()
    env = dict(fp8=G.fp8, X=rnd(5, 256), residual=rnd(5, 256), W=rnd(300, 256), gamma=rnd(256),
               Wg=rnd(384, 256), Wu=rnd(384, 256), Wd=rnd(256, 384))
    exec("\n".join(lines), env)
    torch.cuda.synchronize()
    assert env["Y"].shape == (5, 300) and env["y"].shape == env["h"].shape == (5, 256)


def test_capture_that_forks_and_joins():
    """A captured call whose operands come from two streams, from a copy, and from a fill: it waits for all of
    them at every replay, whatever was left in the buffers."""
    import post_weight_quantization_18_b200 as G
    m, n, k = 70, 640, 1024
    g = torch.Generator().manual_seed(20)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()
    Xs, Ws, Vs = [rnd(m, k) for _ in range(3)], [rnd(n, k) for _ in range(3)], [rnd(n, k) for _ in range(3)]
    X, W, V = torch.empty_like(Xs[0]), torch.empty_like(Ws[0]), torch.empty_like(Vs[0])
    x, w, v = G.fp8.empty(m, k), G.fp8.empty(n, k, 128), G.fp8.empty(n, k, 128)
    hid, copy = G.fp8.empty(m, n), G.fp8.empty(m, n)
    y = torch.empty((m, k), device="cuda")
    down, = _weights(k, n, 21)

    def body(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            G.fp8_quantize(W, w.q, w.scales, 128)
            G.fp8_quantize(V, v.q, v.scales, 128)
        G.fp8_quantize(X, x.q, x.scales)
        main.wait_stream(side)                            # two kernels ahead, one in each stream
        G.fp8_gated_gemm(x.q, x.scales, w.q, w.scales, v.q, v.scales, hid.q, hid.scales)
        copy.q.view(torch.uint8).copy_(hid.q.view(torch.uint8))
        side.wait_stream(main)
        with torch.cuda.stream(side):
            copy.scales.copy_(hid.scales)                 # a copy ahead, in the other stream
        main.wait_stream(side)
        G.fp8_gemm(copy.q, copy.scales, down.q, down.scales, y)
        x.scales.zero_()                                  # a fill behind, and ahead of the next call
        G.fp8_gemm(x.q, x.scales, w.q, w.scales, z)
    z = torch.empty((m, n), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body(torch.cuda.Stream())
    for i in range(12):
        for b in (y, z, hid.scales, copy.scales, w.scales, v.scales):
            b.fill_(float("nan"))
        X.copy_(Xs[i % 3]); W.copy_(Ws[(i + 1) % 3]); V.copy_(Vs[(i + 2) % 3])
        graph.replay()
        torch.cuda.synchronize()
        a = G.fp8.quantize_activations(Xs[i % 3])
        h = G.fp8.gated(a, G.fp8.quantize_weight(Ws[(i + 1) % 3]), G.fp8.quantize_weight(Vs[(i + 2) % 3]))
        torch.cuda.synchronize()
        assert torch.equal(y, G.fp8.linear(h, down, torch.float32)), i
        assert (z == 0).all(), i


def test_calls_from_several_threads():
    """Four threads with a stream each, every size of call among them, first calls of the process included."""
    code = """
import threading, torch, post_weight_quantization_18_b200 as G
sizes = [(1, 512, 2048), (20, 1024, 1024), (50, 4864, 512), (100, 640, 4096), (300, 2048, 512)]
g = torch.Generator().manual_seed(1)
data = [[torch.randn(s, generator=g).bfloat16().cuda() for s in ((m, k), (n, k), (n, k))] for m, n, k in sizes]
out = {}
torch.cuda.synchronize()
def work(t):
    with torch.cuda.stream(torch.cuda.Stream()):
        for i in range(40):
            X, W, V = data[(i + t) % len(data)]
            w, v = G.fp8.quantize_weight(W), G.fp8.quantize_weight(V)
            x, _ = G.fp8.add_rmsnorm(X, None, torch.ones(X.shape[1], device="cuda"))
            h = G.fp8.gated(x, w, v)
            y = G.fp8.linear(x, w)
            out.setdefault((i + t) % len(data), []).append((h.q.view(torch.uint8), h.scales, y))
        torch.cuda.current_stream().synchronize()
ts = [threading.Thread(target=work, args=(t,)) for t in range(4)]
[t.start() for t in ts]; [t.join() for t in ts]
torch.cuda.synchronize()
n = 0
for i, (X, W, V) in enumerate(data):
    want = out[i][0]
    assert torch.isfinite(want[2]).all()
    for got in out[i]:
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i
        n += 1
print(n)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "160", r.stdout + r.stderr
