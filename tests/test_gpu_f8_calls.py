"""The e4m3 operators as a program calls them: one after the other, captured, on several streams, far apart in memory, refused."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib
from oracle import attn_oracle as A
from oracle import f8_oracle as F
from tests.helpers import bits16, f64
from tests.test_gpu_f8 import byts, check_codes, held, matrix, random_matrix, sum_tolerance, swiglu_tolerance, values

pytestmark = pytest.mark.gpu

U8 = torch.uint8
# sizes that take each of the kernels: few rows, a batch, many
SHAPES = [(3, 640, 1152), (70, 640, 1152), (2100, 640, 1152)]


def dense(dev, rng, rows, cols, size=1.0):
    """bf16 weights, quantised."""
    w = torch.from_numpy(size * rng.standard_normal((rows, cols)) / np.sqrt(cols)).bfloat16().to(dev)
    return lib.bgq_f8_quantise(w, block_rows=128)


@pytest.mark.parametrize("first,m", [(0, 150), (150, 1), (151, 40)])
def test_a_decoder_layer(cuda_device, first, m):
    """A layer's dense path around attention, from the residual in front of it to the one behind its feed-forward block, for a prompt, a
    token and a chunk: every step against the oracle on what the step before it gave."""
    dev, rng = cuda_device, np.random.default_rng(17 + first)
    d, hq, hkv, hd, f, page = 512, 4, 2, 128, 768, 16
    heads = hq + 2 * hkv
    Wqkv, Wo = dense(dev, rng, heads * hd, d), dense(dev, rng, d, hq * hd)
    G, U, D = dense(dev, rng, f, d), dense(dev, rng, f, d), dense(dev, rng, d, f)
    rho = [torch.from_numpy(1 + 0.1 * rng.standard_normal(d)).bfloat16().to(dev) for _ in range(3)]
    h = torch.from_numpy(rng.standard_normal((m, d))).float().to(dev)
    plan, cache = lib.RopePlan(hd, hd, 1e4, [hd // 2]), lib.KV4Cache.empty(64, hkv, page, hd, device=dev)
    pages = torch.arange(63, -1, -1, dtype=torch.int32, device=dev).view(1, 64)
    past = torch.from_numpy(rng.standard_normal((2, max(first, 1), hkv, hd))).bfloat16().to(dev)
    if first:
        seqs = lib.KV4Seqs(torch.tensor([first], dtype=torch.int32, device=dev), rows=first, pages=pages, max_q=first,
                           q_start=torch.tensor([0, first], dtype=torch.int32, device=dev))
        lib.bgq_kv4_append(cache, seqs, past[0], past[1])
    seqs = lib.KV4Seqs(torch.tensor([first + m], dtype=torch.int32, device=dev), rows=m, pages=pages, max_q=m,
                       q_start=torch.tensor([0, m], dtype=torch.int32, device=dev))
    h0 = h.clone()
    x0, _ = lib.bgq_rmsnorm_f8(h, rho[0], 1e-6)
    qkv, _ = lib.bgq_f8_gemm(Wqkv, x0)
    turned = qkv.clone().view(m, heads, hd)
    lib.bgq_rope(plan, turned[:, :hq + hkv], torch.arange(first, first + m, dtype=torch.int32, device=dev), y=turned[:, :hq + hkv])
    lib.bgq_kv4_append(cache, seqs, turned[:, hq:hq + hkv], turned[:, hq + hkv:])
    o, _ = lib.bgq_kv4_attention(cache, seqs, turned[:, :hq])
    xo = lib.bgq_f8_quantise(o.view(m, hq * hd))
    _, attn = lib.bgq_f8_gemm(Wo, xo, want_out=False, want_f32=True)
    x1, _ = lib.bgq_rmsnorm_f8(h, rho[1], 1e-6, delta=attn)
    h1 = h.clone()
    act, _ = lib.bgq_f8_swiglu(G, U, x1)
    ffn, _ = lib.bgq_f8_gemm(D, act)
    x2, a2 = lib.bgq_rmsnorm_f8(h, rho[2], 1e-6, delta=ffn, want_a=True)
    torch.cuda.synchronize()

    def norm(x, hh, r):
        ref = F.norm(f64(hh), None, f64(r), 1e-6)[1]
        check_codes(x, ref, np.abs(ref) * 60 * 2.0 ** -24 + 2.0 ** -149)

    def gemm(y, W, x):
        ref, size = F.product(values(x), values(W))
        tol = sum_tolerance(size, x.cols)
        assert (np.abs(f64(y) - ref) <= tol + (0 if y.dtype == torch.float32 else (np.abs(ref) + tol) * 2.0 ** -8)).all()

    norm(x0, h0, rho[0])
    gemm(qkv, Wqkv, x0)
    arrays = [t.cpu().numpy().view(np.uint32) if t.dtype == torch.int32 else bits16(t) for t in (cache.k_q, cache.k_sb, cache.v_q, cache.v_sb)]
    ref = A.kv4_attention(arrays, [first + m], [0, m], m, pages.cpu().numpy(), f64(turned[:, :hq]), hd ** -0.5)[0]
    assert np.linalg.norm(f64(o) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    q, s = F.quantise(f64(o).reshape(m, -1))
    assert np.array_equal(byts(xo.q), q) and np.array_equal(byts(xo.scale), s)
    gemm(attn, Wo, xo)
    assert torch.equal(h1, h0 + attn)
    norm(x1, h1, rho[1])
    (g, sg), (u, su) = F.product(values(x1), values(G)), F.product(values(x1), values(U))
    check_codes(act, F.swiglu(g, u), swiglu_tolerance(g, u, sg, su, d))
    gemm(ffn, D, act)
    assert torch.equal(h, h1 + ffn.float())
    norm(x2, h, rho[2])
    ref = F.norm(f64(h), None, f64(rho[2]), 1e-6)[1]
    assert (np.abs(f64(a2) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -17)).all()


def chain(dev, rng, m, n, k):
    """A step as a program runs it, over buffers of its own: (buffers to fill, the call, what it gives)."""
    h, delta = torch.empty(m, k, device=dev), torch.empty(m, k, dtype=torch.bfloat16, device=dev)
    x, act = lib.F8Matrix.empty(m, k, device=dev), lib.F8Matrix.empty(m, n, device=dev)
    G, U, D = dense(dev, rng, n, k), dense(dev, rng, n, k), dense(dev, rng, k, n)
    y, ws = torch.empty(m, k, device=dev), lib.workspace(256, dev)

    def call():
        lib.bgq_rmsnorm_f8(h, None, 1e-6, delta=delta, out=x)
        lib.bgq_f8_swiglu(G, U, x, h=act, ws=ws)
        lib.bgq_f8_gemm(D, act, out_f32=y, ws=ws)

    def fill(seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        h.copy_(torch.randn(m, k, generator=g, device=dev))
        delta.copy_(torch.randn(m, k, generator=g, device=dev))

    return fill, call, y, ws


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_captured_and_replayed(cuda_device, m, n, k):
    rng = np.random.default_rng(m)
    fill, call, y, ws = chain(cuda_device, rng, m, n, k)
    want = []
    for seed in range(3):
        fill(seed)
        call()
        want.append(y.clone())
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        call()
    for turn in range(2):
        for seed in range(3):
            fill(seed)
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[seed])
    assert not torch.equal(want[0], want[1])
    assert lib.read_device_status(ws) == lib.OK


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from bit_group_quantized_gb300 import lib
m, n, k, dev = {m}, 640, 1152, torch.device("cuda")
h, x, act = torch.randn(m, k, device=dev), lib.F8Matrix.empty(m, k), lib.F8Matrix.empty(m, n)
w, W, V = torch.randn(n, k, device=dev).bfloat16(), lib.F8Matrix.empty(n, k, 128), lib.F8Matrix.empty(k, n, 128)
y, ws = torch.zeros(m, k, device=dev), lib.workspace(256, dev)
def call():
    lib.bgq_f8_quantise(w, out=W)
    lib.bgq_f8_quantise(w.view(k, n), out=V)
    lib.bgq_rmsnorm_f8(h, None, 1e-6, out=x)
    lib.bgq_f8_swiglu(W, W, x, h=act, ws=ws)
    lib.bgq_f8_gemm(V, act, out_f32=y, ws=ws)
torch.cuda.synchronize()
s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
    call()
g.replay()
torch.cuda.synchronize()
got = y.clone()
y.zero_()
call()
torch.cuda.synchronize()
assert torch.equal(got, y) and bool(torch.isfinite(y).all()) and float(y.abs().max()) > 0
"""


@pytest.mark.parametrize("m", [3, 70, 2100])
def test_the_first_call_of_a_process_captured(cuda_device, m):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, m=m)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_graphs_and_streams_share_a_workspace(cuda_device):
    """Two captured steps of different sizes, replayed on two streams at once over one workspace, beside direct calls on a third."""
    dev = cuda_device
    steps = [chain(dev, np.random.default_rng(5 + i), *s) for i, s in enumerate(SHAPES)]
    want = []
    for fill, call, y, _ in steps:
        fill(7)
        call()
        want.append(y.clone())
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in steps], []
    for (_, call, _, _), s in zip(steps[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            call()
        graphs.append(g)
    for turn in range(20):
        for fill, _, y, _ in steps:
            fill(7)
            y.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            steps[2][1]()
        torch.cuda.synchronize()
        for (_, _, y, _), w in zip(steps, want):
            assert torch.equal(y, w), turn


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_weights_and_inputs_of_the_call_before(cuda_device, m, n, k):
    """Weights quantised, and inputs written, by the calls just before on the same stream, again and again into the same memory."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(m)
    w = [torch.randn(n, k, generator=g, device=dev).bfloat16() for _ in range(4)]
    x = [torch.randn(m, k, generator=g, device=dev).bfloat16() for _ in range(4)]
    want = [lib.bgq_f8_gemm(lib.bgq_f8_quantise(a, block_rows=128), lib.bgq_f8_quantise(b))[0] for a, b in zip(w, x)]
    torch.cuda.synchronize()
    W, X, ws = lib.F8Matrix.empty(n, k, 128, dev), lib.F8Matrix.empty(m, k, 1, dev), lib.workspace(256, dev)
    got = [torch.empty_like(want[0]) for _ in range(40)]
    for i, y in enumerate(got):
        if i % 8 < 4:
            lib.bgq_f8_quantise(x[i % 4], out=X)
            lib.bgq_f8_quantise(w[i % 4], out=W)
        else:
            lib.bgq_f8_quantise(w[i % 4], out=W)
            lib.bgq_f8_quantise(x[i % 4], out=X)
        lib.bgq_f8_gemm(W, X, out=y, ws=ws)
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4]), i


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_on_a_given_stream(cuda_device, m, n, k):
    rng = np.random.default_rng(m + 1)
    W, _ = random_matrix(cuda_device, rng, n, k, 128)
    X, _ = random_matrix(cuda_device, rng, m, k, 1)
    h = torch.from_numpy(rng.standard_normal((m, k))).float().to(cuda_device)
    want, (x0, a0) = lib.bgq_f8_gemm(W, X)[0], lib.bgq_rmsnorm_f8(h.clone(), None, 1e-6, want_a=True)
    q0, s0 = lib.bgq_f8_swiglu(W, W, X)[0], lib.bgq_f8_quantise(a0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lib.bgq_f8_gemm(W, X, stream=s)[0]
    x1, a1 = lib.bgq_rmsnorm_f8(h, None, 1e-6, want_a=True, stream=s)
    q1, s1 = lib.bgq_f8_swiglu(W, W, X, stream=s)[0], lib.bgq_f8_quantise(a1, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(a0, a1)
    for a, b in ((x0, x1), (q0, q1), (s0, s1)):
        assert all(np.array_equal(u, v) for u, v in zip(held(a), held(b)))


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_a_row_does_not_depend_on_the_others(cuda_device, m, n, k):
    rng = np.random.default_rng(m + 2)
    W, _ = random_matrix(cuda_device, rng, n, k, 128, lo=116, hi=119)
    X, _ = random_matrix(cuda_device, rng, m, k, 1, lo=116, hi=119)
    y, (h, _) = lib.bgq_f8_gemm(W, X)[0], lib.bgq_f8_swiglu(W, W, X)
    q, s = held(h)
    keep = m // 2
    X.q.view(U8)[:keep] = 0x7f
    X.q.view(U8)[keep + 1:] = 0x7e
    X.scale.view(U8)[keep + 1:] = 160
    y2, (h2, _) = lib.bgq_f8_gemm(W, X)[0], lib.bgq_f8_swiglu(W, W, X)
    q2, s2 = held(h2)
    assert torch.equal(y[keep], y2[keep]) and np.array_equal(q[keep], q2[keep]) and np.array_equal(s[keep], s2[keep])


@pytest.mark.parametrize("m", [5, 40, 600])
def test_rows_beyond_32_bits(cuda_device, m):
    """Codes, inputs and results whose rows lie so far apart that their places pass 2^32."""
    dev, rng, k, n = cuda_device, np.random.default_rng(m), 272, 144
    far = (5 << 30) // m // 256 * 256
    q = torch.zeros(m * far, dtype=U8, device=dev)
    x = rng.standard_normal((m, k))
    xb = torch.from_numpy(x).bfloat16().to(dev)
    X = lib.F8Matrix(torch.as_strided(q.view(lib._F8), (m, k), (far, 1)),
                     lib.F8Matrix.empty_scale(m, k, dev))
    lib.bgq_f8_quantise(xb, out=X)
    near = lib.bgq_f8_quantise(xb)
    assert torch.equal(X.q.contiguous().view(U8), near.q.view(U8))
    W, _ = random_matrix(dev, rng, n, k, 128, lo=116, hi=119)
    want, (h, _) = lib.bgq_f8_gemm(W, near, want_f32=True), lib.bgq_f8_swiglu(W, W, near)
    got, (h2, _) = lib.bgq_f8_gemm(W, X, want_f32=True), lib.bgq_f8_swiglu(W, W, X)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(np.array_equal(a, b) for a, b in zip(held(h), held(h2)))
    # results and the quantiser's input as far apart, in the same memory
    y = torch.as_strided(q.view(torch.bfloat16), (m, n), (far // 2, 1))
    lib.bgq_f8_gemm(W, near, out=y)
    assert torch.equal(y, want[0])
    wide = torch.as_strided(q.view(torch.bfloat16), (m, k), (far // 2, 1))
    wide.copy_(xb)
    again = lib.bgq_f8_quantise(wide)
    assert all(np.array_equal(a, b) for a, b in zip(held(again), held(near)))
    H = lib.F8Matrix(torch.as_strided(q.view(lib._F8), (m, n), (far, 1)), lib.F8Matrix.empty_scale(m, n, dev))
    lib.bgq_f8_swiglu(W, W, near, h=H)
    assert torch.equal(H.q.contiguous().view(U8), h.q.view(U8)) and np.array_equal(byts(H.scale), byts(h.scale))


def test_two_million_narrow_rows(cuda_device):
    """Rows counted beyond 16 bits of everything, 16 columns each."""
    dev, m, k, n = cuda_device, 65535 * 32 + 37, 16, 16
    W, w = random_matrix(dev, np.random.default_rng(1), n, k, 128)
    q = torch.randint(0, 127, (m, k), dtype=U8, device=dev, generator=torch.Generator(device=dev).manual_seed(2))
    s = torch.full((m, 4), 127, dtype=U8, device=dev)
    X = lib.F8Matrix(q.view(lib._F8), s.view(lib._E8)[:, :1])
    y = lib.bgq_f8_gemm(W, X, want_out=False, want_f32=True)[1]
    h, _ = lib.bgq_f8_swiglu(W, W, X)
    for rows in (slice(0, 64), slice(65535 * 32 - 40, m)):
        x = F.values(q[rows].cpu().numpy(), np.full((len(range(*rows.indices(m))), 1), 127, dtype=np.uint8))
        ref, size = F.product(x, w)
        assert (np.abs(f64(y[rows]) - ref) <= sum_tolerance(size, k)).all()
        part = lib.F8Matrix(h.q[rows], h.scale[rows])
        check_codes(part, F.swiglu(ref, ref), swiglu_tolerance(ref, ref, size, size, k))


def test_no_rows(cuda_device):
    dev = cuda_device
    W, _ = random_matrix(dev, np.random.default_rng(1), 128, 256, 128)
    X = lib.F8Matrix.empty(0, 256, device=dev)
    assert lib.bgq_f8_gemm(W, X)[0].shape == (0, 128)
    assert lib.bgq_f8_swiglu(W, W, X)[0].q.shape == (0, 128)
    assert lib.bgq_rmsnorm_f8(torch.empty(0, 256, device=dev), None, 1e-6)[0].rows == 0
    assert lib.bgq_f8_quantise(torch.empty(0, 256, dtype=torch.bfloat16, device=dev)).rows == 0


def test_what_the_binding_refuses(cuda_device):
    dev = cuda_device
    W, _ = random_matrix(dev, np.random.default_rng(1), 128, 256, 128)
    X, _ = random_matrix(dev, np.random.default_rng(2), 8, 256, 1)
    q, s = torch.zeros(8, 256, dtype=U8, device=dev), torch.zeros(8, 4, dtype=U8, device=dev)
    f8, e8 = q.view(lib._F8), s.view(lib._E8)[:, :2]
    h, x = torch.zeros(8, 256, device=dev), torch.zeros(8, 256, dtype=torch.bfloat16, device=dev)
    bad = [
        lambda: lib.F8Matrix(q, e8), lambda: lib.F8Matrix(f8, s[:, :2]), lambda: lib.F8Matrix(f8, e8[:7]), lambda: lib.F8Matrix(f8, e8, 64),
        lambda: lib.F8Matrix(f8[:, ::2], e8[:, :1]), lambda: lib.F8Matrix(f8, e8.cpu()), lambda: lib.F8Matrix(f8.T, e8),
        lambda: lib.F8Matrix(f8, torch.zeros(16, dtype=U8, device=dev).view(lib._E8).view(8, 2)),
        lambda: lib.F8Matrix.empty(8, 250, device=dev), lambda: lib.F8Matrix.empty(8, 256, 2, device=dev),
        lambda: lib.bgq_f8_quantise(h), lambda: lib.bgq_f8_quantise(x, out=W), lambda: lib.bgq_f8_quantise(x[:, ::2]), lambda: lib.bgq_f8_quantise(None),
        lambda: lib.bgq_rmsnorm_f8(x, None, 1e-6), lambda: lib.bgq_rmsnorm_f8(h, x[0], 1e-6, delta=x[:4]), lambda: lib.bgq_rmsnorm_f8(h, h[0], 1e-6),
        lambda: lib.bgq_rmsnorm_f8(h[:, :128], None, 1e-6), lambda: lib.bgq_rmsnorm_f8(h, None, -1.0), lambda: lib.bgq_rmsnorm_f8(h, None, 1e-6, out=W),
        lambda: lib.bgq_rmsnorm_f8(h, None, 1e-6, a=h), lambda: lib.bgq_rmsnorm_f8(h, None, 1e-6, delta=x.cpu()),
        lambda: lib.bgq_f8_gemm(X, X), lambda: lib.bgq_f8_gemm(W, W), lambda: lib.bgq_f8_gemm(W, x), lambda: lib.bgq_f8_gemm(W, X, out=x),
        lambda: lib.bgq_f8_gemm(W, X, out=torch.empty(8, 128, device=dev)), lambda: lib.bgq_f8_gemm(W, X, want_out=False),
        lambda: lib.bgq_f8_gemm(W, X, out=torch.empty(8, 132, dtype=torch.bfloat16, device=dev)[:, :128]),
        lambda: lib.bgq_f8_gemm(W, X, ws=torch.zeros(64, dtype=U8, device=dev)), lambda: lib.bgq_f8_gemm(W, X, ws=torch.zeros(256, dtype=U8)),
        lambda: lib.bgq_f8_gemm(W, X, out=torch.empty(8, 128, dtype=torch.bfloat16, device=dev), out_f32=torch.empty(8, 136, device=dev)[:, :128]),
        lambda: lib.bgq_f8_swiglu(W, X, X), lambda: lib.bgq_f8_swiglu(W, W, X, h=X), lambda: lib.bgq_f8_swiglu(W, W, X, want_h=False),
        lambda: lib.bgq_f8_swiglu(W, W, X, out=h), lambda: lib.bgq_f8_swiglu(W, None, X),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(lib.BGQError):
            call()
            pytest.fail(f"call {i} was not refused")
