"""The e4m3 operators on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic:
* a quantiser of bf16 values makes the oracle's codes and scales: scaling by a power of two is exact;
* fp32 sums: each of n additions is off by at most 2^-23 of a partial sum's size (the tensor cores cut, 2^-24 otherwise),
  which the sum of the terms' sizes bounds;
* a result rounded once: 2^-8 of a bf16 value, 2^-4 of an e4m3 value (2^-10 scales where it is subnormal).
"""

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib
from oracle import bgq_oracle as O
from oracle import f8_oracle as F
from tests.helpers import bits16, f64

pytestmark = pytest.mark.gpu

U8 = torch.uint8


def byts(t):
    return t.detach().view(U8).cpu().numpy()


def held(m: lib.F8Matrix):
    return byts(m.q), byts(m.scale)


def values(m: lib.F8Matrix):
    return F.values(*held(m), m.block_rows)


def matrix(dev, q, s, block_rows, q_pad=0, s_pad=0, q_dirt=0x7f):
    """An F8Matrix of these bytes whose rows lie q_pad and s_pad bytes further apart; NaN codes in between."""
    rows, cols = q.shape
    wide = torch.full((max(rows, 1), cols + q_pad), q_dirt, dtype=U8, device=dev)
    wide[:rows, :cols] = torch.from_numpy(q).to(dev)
    n = s.shape[1]
    sw = torch.full((max(s.shape[0], 1), -(-n // 4) * 4 + s_pad), 200, dtype=U8, device=dev)
    sw[:s.shape[0], :n] = torch.from_numpy(s).to(dev)
    return lib.F8Matrix(wide.view(lib._F8)[:rows, :cols], sw.view(lib._E8)[:s.shape[0], :n], block_rows)


def random_matrix(dev, rng, rows, cols, block_rows, lo=124, hi=131, **pads):
    """Codes of all sizes (no NaN) and scales of different sizes side by side."""
    q = rng.integers(0, 127, (rows, cols)).astype(np.uint8) | (rng.integers(0, 2, (rows, cols)).astype(np.uint8) << 7)
    s = rng.integers(lo, hi, (-(-rows // block_rows), -(-cols // F.BLOCK))).astype(np.uint8)
    return matrix(dev, q, s, block_rows, **pads), F.values(q, s, block_rows)


def check_codes(m: lib.F8Matrix, ref, off, what=""):
    """The codes and scales of values that are `off` from ref at most."""
    q, s = held(m)
    for j in range(s.shape[1]):
        a, o = np.abs(ref[:, j * 128:(j + 1) * 128]), off[:, j * 128:(j + 1) * 128]
        least, most = np.max(a - o, 1), np.max(a + o, 1)
        scale = 2.0 ** (s[:, j].astype(np.float64) - 127)
        assert (least <= 448 * scale).all(), (what, j)
        assert ((most > 224 * scale) | (s[:, j] == 0)).all(), (what, j)
    step = np.repeat(2.0 ** (s.astype(np.float64) - 127), 128, 1)[:, :ref.shape[1]]
    got = F.values(q, s)
    tol = off + np.maximum((np.abs(ref) + off) * 2.0 ** -4, step * 2.0 ** -10)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("rows,cols,pad,block", [
    (1, 16, 0, 1), (1, 128, 0, 1), (3, 144, 8, 1), (2, 256, 0, 1), (37, 1040, 16, 1), (5, 4096, 0, 1), (1, 65536, 0, 1),
    (301, 272, 0, 1), (1, 16, 0, 128), (128, 128, 0, 128), (129, 144, 24, 128), (300, 1040, 0, 128), (127, 4096, 8, 128)])
def test_quantise(cuda_device, rows, cols, pad, block):
    rng = np.random.default_rng(rows * 7 + cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols + pad)) * np.exp(3 * rng.standard_normal((rows, 1)))).bfloat16()
    if pad:
        x[:, cols:] = float("nan")  # between the rows
    m = lib.bgq_f8_quantise(x.to(cuda_device)[:, :cols], block_rows=block)
    q, s = F.quantise(f64(x[:, :cols]), block)
    assert np.array_equal(byts(m.scale), s)
    assert np.array_equal(byts(m.q), q)


@pytest.mark.parametrize("block", [1, 128])
def test_quantise_special_values(cuda_device, block):
    """Every finite bf16 value beside each power of two's neighbours; zeros, NaN and infinities, which stay in their block."""
    bits = np.arange(0x7f80, dtype=np.uint16)
    every = O.bf16_to_f64(np.concatenate([bits, bits | 0x8000, np.zeros(-2 * len(bits) % 128, dtype=np.uint16)])).reshape(-1, 128)
    tops = np.zeros((256, 128))
    tops[:254, 0] = 2.0 ** (np.arange(254) - 126.0)
    edge = np.zeros((6, 128))
    edge[0, 7], edge[1, 7], edge[2, 7] = 448.0, -450.0, 446.0  # 450 is 448's neighbour in bf16
    edge[3, :], edge[4, 5], edge[5, 127] = -0.0, 2.0 ** -133, -(2.0 ** -126)
    x = np.concatenate([every, tops, edge])
    x = np.tile(x, (1, 3))
    if block > 1:  # rows of one kind of size together: the largest of a block decides for all of it
        x = np.repeat(x[:: max(1, len(x) // 40)], 128, 0)
    x[5 * block, 130], x[6 * block, 200], x[7 * block, 383] = np.nan, np.inf, -np.inf
    t = torch.from_numpy(x).bfloat16()
    m = lib.bgq_f8_quantise(t.to(cuda_device), block_rows=block)
    q, s = F.quantise(f64(t), block)
    assert np.array_equal(byts(m.scale), s)
    assert np.array_equal(byts(m.q), q)
    bad = np.isnan(values(m))
    assert bad[5 * block, 128:256].all() and not bad[5 * block, :128].any() and not bad[5 * block, 256:].any()


# ----------------------------------------------------------------------- norm
def check_norm(dev, batch, d, f32, rho, eps=1e-6, size=1.0, seed=0):
    rng = np.random.default_rng(seed + batch * 3 + d)
    h = torch.from_numpy(size * 3 * rng.standard_normal((batch, d)) * np.exp(rng.standard_normal(d))).float()
    delta = None if f32 is None else torch.from_numpy(size * rng.standard_normal((batch, d))).to(torch.float32 if f32 else torch.bfloat16)
    r = torch.from_numpy(1 + 0.2 * rng.standard_normal(d)).bfloat16() if rho else None
    hd = h.to(dev)
    m, a = lib.bgq_rmsnorm_f8(hd, None if r is None else r.to(dev), eps, delta=None if delta is None else delta.to(dev), want_a=True)
    want = h if delta is None else h + delta.float()
    assert torch.equal(hd.cpu(), want)  # one fp32 addition
    _, ref = F.norm(want.double().numpy(), None, None if r is None else f64(r), eps)
    # a row's squares: at most 64 + 5 + 32 additions of 2^-24 each, half of that through the root, and five more roundings
    off = np.abs(ref) * 60 * 2.0 ** -24 + 2.0 ** -149
    assert (np.abs(f64(a) - ref) <= off + np.abs(ref) * 2.0 ** -8 + 2.0 ** -134).all()
    check_codes(m, ref, off)


@pytest.mark.parametrize("batch,d", [(1, 16), (1, 128), (2, 144), (3, 1024), (5, 1040), (64, 4096), (7, 2048), (3, 5008), (2, 16384),
                                     (2, 16400), (1, 65536), (1000, 256)])
@pytest.mark.parametrize("f32", [None, False, True])
def test_norm(cuda_device, batch, d, f32):
    check_norm(cuda_device, batch, d, f32, rho=f32 is not None)


@pytest.mark.parametrize("size", [1e-15, 1e15])
def test_norm_of_small_and_large_rows(cuda_device, size):
    check_norm(cuda_device, 3, 4096, False, True, size=size)


def test_norm_zeros_nan_and_infinities(cuda_device):
    h = torch.zeros(4, 640)
    h[1, 300], h[2, 5], h[3] = float("nan"), float("inf"), 1.0
    m, a = lib.bgq_rmsnorm_f8(h.to(cuda_device), None, 1e-6, want_a=True)
    v = values(m)
    assert (v[0] == 0).all() and (byts(m.scale)[0] == 0).all()
    assert np.isnan(v[1]).all()
    assert np.isnan(v[2, :128]).all() and (v[2, 128:] == 0).all()
    assert np.abs(v[3] - 1).max() <= 2.0 ** -4


# -------------------------------------------------------------------- product
def sum_tolerance(size, k):
    """Of a sum of k products: a step for every 32 columns, and 16 for the scales and the parts."""
    return size * (k / 32 + 16) * 2.0 ** -23


def check_gemm(dev, m, n, k, seed=0, pads=None, **scales):
    rng = np.random.default_rng(seed + m * 31 + n * 7 + k)
    pads = pads or {}
    W, w = random_matrix(dev, rng, n, k, 128, **scales, **pads)
    X, x = random_matrix(dev, rng, m, k, 1, **scales, **pads)
    ref, size = F.product(x, w)
    y, yf = lib.bgq_f8_gemm(W, X, want_f32=True)
    tol = sum_tolerance(size, k)
    assert (np.abs(f64(yf) - ref) <= tol).all(), np.abs(f64(yf) - ref).max()
    assert torch.equal(y, yf.bfloat16())
    one, none = lib.bgq_f8_gemm(W, X)
    assert none is None and torch.equal(one, y)


SIZES = [(1, 16, 16), (1, 1, 128), (1, 128, 144), (2, 17, 256), (8, 130, 512), (9, 300, 640), (16, 144, 1040), (17, 256, 384), (31, 257, 1024),
         (33, 128, 4096), (64, 1000, 2064), (65, 96, 128), (127, 272, 272), (128, 128, 128), (129, 129, 144), (200, 512, 1536), (255, 384, 4112),
         (257, 520, 1168), (300, 1000, 640), (513, 260, 144), (700, 1296, 2048), (1025, 777, 16), (2600, 2064, 528), (4100, 5003, 128), (2100, 16, 256), (2050, 1, 128), (40, 3, 128), (40, 100, 16), (300, 260, 112),
         (2100, 700, 64)]
# tiles of 192 (one and three of a pair of CTAs), 160 and 128 rows of W
NARROW = [(2100, 1187, 2064), (4600, 2300, 2064), (2100, 2301, 640), (2100, 1000, 2064)]


@pytest.mark.parametrize("m,n,k", SIZES + NARROW)
def test_gemm(cuda_device, m, n, k):
    check_gemm(cuda_device, m, n, k)


@pytest.mark.parametrize("m", [1, 40, 300, 1500])
def test_gemm_rows_apart(cuda_device, m):
    check_gemm(cuda_device, m, 200, 656, pads=dict(q_pad=48, s_pad=4))


def test_gemm_scales_at_the_ends(cuda_device):
    """Scales whose product leaves fp32 on its way, and results that do not."""
    dev, k = cuda_device, 256
    for m in (3, 70, 300):
        q = np.full((m, k), 0x38, dtype=np.uint8)  # 1
        w = np.full((130, k), 0x38, dtype=np.uint8)
        for ex, ew in ((0, 254), (254, 0), (7, 247), (127, 127), (20, 120), (200, 150), (1, 160)):
            X = matrix(dev, q, np.full((m, 2), ex, dtype=np.uint8), 1)
            W = matrix(dev, w, np.full((2, 2), ew, dtype=np.uint8), 128)
            yf = lib.bgq_f8_gemm(W, X, want_out=False, want_f32=True)[1]
            assert (f64(yf) == k * 2.0 ** (ex + ew - 254)).all(), (m, ex, ew, yf[0, 0])


@pytest.mark.parametrize("m", [5, 40, 300, 1200])
def test_gemm_nan_stays_in_its_row(cuda_device, m):
    rng = np.random.default_rng(m)
    W, w = random_matrix(cuda_device, rng, 150, 400, 128)
    X, x = random_matrix(cuda_device, rng, m, 400, 1)
    X.q.view(U8)[2, 399] = 0xff
    W.q.view(U8)[140, 0] = 0x7f
    y = f64(lib.bgq_f8_gemm(W, X)[0])
    assert np.isnan(y[2]).all() and np.isnan(y[:, 140]).all()
    y[2], y[:, 140] = 0, 0
    assert np.isfinite(y).all()


@pytest.mark.parametrize("m", [4, 100, 600])
def test_gemm_writes_its_rows_alone(cuda_device, m):
    rng = np.random.default_rng(m)
    W, _ = random_matrix(cuda_device, rng, 133, 272, 128)
    X, _ = random_matrix(cuda_device, rng, m, 272, 1)
    wide = torch.full((m + 2, 160), -7.0, dtype=torch.bfloat16, device=cuda_device)
    widef = torch.full((m + 2, 160), -7.0, device=cuda_device)
    lib.bgq_f8_gemm(W, X, out=wide[1:m + 1, :133], out_f32=widef[1:m + 1, :133])
    ref = lib.bgq_f8_gemm(W, X, want_f32=True)
    for got, want in ((wide, ref[0]), (widef, ref[1])):
        assert torch.equal(got[1:m + 1, :133], want)
        assert (got[:, 133:] == -7).all() and (got[0] == -7).all() and (got[m + 1] == -7).all()


# --------------------------------------------------------------------- gated
def swiglu_tolerance(g, u, size_g, size_u, k):
    """Of silu(g) u: silu's slope is at most 1.1, the exponential is off by 2 + 1.2 |g| units of 2^-23 (it has no part in the result
    where it overflows), the reciprocal and three products by one each."""
    eg, eu = sum_tolerance(size_g, k), sum_tolerance(size_u, k)
    silu = np.abs(F.swiglu(g, 1.0))
    return 1.1 * eg * (np.abs(u) + eu) + (silu + 1.1 * eg) * eu + silu * np.abs(u) * (8 + 1.2 * np.minimum(np.abs(g), 89)) * 2.0 ** -23 + 2.0 ** -126 * np.abs(u)


def check_swiglu(dev, m, n, k, seed=0, pads=None):
    rng = np.random.default_rng(seed + m * 31 + n * 7 + k)
    pads = pads or {}
    lo = 122 - int(np.log2(k) / 2)  # gates of a few units: codes are some 30 large
    G, g = random_matrix(dev, rng, n, k, 128, lo=lo - 3, hi=lo, **pads)
    U, u = random_matrix(dev, rng, n, k, 128, lo=lo - 1, hi=lo + 2, **pads)
    X, x = random_matrix(dev, rng, m, k, 1, lo=119, hi=122, **pads)
    (g, sg), (u, su) = F.product(x, g), F.product(x, u)
    ref, off = F.swiglu(g, u), swiglu_tolerance(g, u, sg, su, k)
    h, y = lib.bgq_f8_swiglu(G, U, X, want_out=True)
    assert (np.abs(f64(y) - ref) <= off + (np.abs(ref) + off) * 2.0 ** -8 + 2.0 ** -134).all()
    check_codes(h, ref, off)
    alone, none = lib.bgq_f8_swiglu(G, U, X)
    assert none is None and torch.equal(alone.q.view(U8), h.q.view(U8)) and torch.equal(alone.scale.view(U8), h.scale.view(U8))
    none, alone = lib.bgq_f8_swiglu(G, U, X, want_h=False, want_out=True)
    assert none is None and torch.equal(alone, y)


@pytest.mark.parametrize("m,n,k", [(m, -(-n // 16) * 16, k) for m, n, k in SIZES])
def test_swiglu(cuda_device, m, n, k):
    check_swiglu(cuda_device, m, n, k)


@pytest.mark.parametrize("m", [1, 40, 300, 1500])
def test_swiglu_rows_apart(cuda_device, m):
    check_swiglu(cuda_device, m, 208, 656, pads=dict(q_pad=48, s_pad=4))


@pytest.mark.parametrize("m", [4, 100, 600])
def test_swiglu_writes_its_rows_alone(cuda_device, m):
    rng = np.random.default_rng(m)
    G, _ = random_matrix(cuda_device, rng, 144, 272, 128, lo=116, hi=119)
    U, _ = random_matrix(cuda_device, rng, 144, 272, 128, lo=116, hi=119)
    X, _ = random_matrix(cuda_device, rng, m, 272, 1, lo=116, hi=119)
    q = torch.full((m + 2, 160), 0x55, dtype=U8, device=cuda_device)
    s = torch.full((m + 2, 8), 0x55, dtype=U8, device=cuda_device)
    h = lib.F8Matrix(q.view(lib._F8)[1:m + 1, :144], s.view(lib._E8)[1:m + 1, :2])
    lib.bgq_f8_swiglu(G, U, X, h=h)
    ref, _ = lib.bgq_f8_swiglu(G, U, X)
    assert torch.equal(q[1:m + 1, :144], ref.q.view(U8)) and torch.equal(s[1:m + 1, :2], ref.scale.view(U8))
    assert (q[:, 144:] == 0x55).all() and (q[0] == 0x55).all() and (q[m + 1] == 0x55).all()
    assert (s[:, 2:] == 0x55).all() and (s[0] == 0x55).all() and (s[m + 1] == 0x55).all()


@pytest.mark.parametrize("m", [3, 90, 400])
def test_swiglu_blocks_that_are_not_finite(cuda_device, m):
    """A NaN makes its row's block of 128 NaN, and no other; a block of zeros has zeros."""
    rng = np.random.default_rng(m)
    G, _ = random_matrix(cuda_device, rng, 272, 128, 128, lo=116, hi=119)
    U, _ = random_matrix(cuda_device, rng, 272, 128, 128, lo=116, hi=119)
    X, _ = random_matrix(cuda_device, rng, m, 128, 1, lo=116, hi=119)
    U.q.view(U8)[130, 3] = 0x7f  # NaN for all rows, in the second block
    X.q.view(U8)[1] = 0
    X.q.view(U8)[1, 3] = 0x7f    # NaN everywhere
    X.q.view(U8)[2, :] = 0
    h, _ = lib.bgq_f8_swiglu(G, U, X)
    v = values(h)
    assert np.isnan(v[:, 128:256]).all() and np.isnan(v[1]).all()
    assert (v[2, :128] == 0).all() and (v[2, 256:] == 0).all()
    assert np.isfinite(v[0, :128]).all() and np.isfinite(v[0, 256:]).all()


@pytest.mark.parametrize("m", [2, 40, 500])
def test_swiglu_of_far_negative_gates(cuda_device, m):
    """silu(-88) is below fp32's normal numbers, its product with a large up is not."""
    k, n = 256, 144
    q = np.zeros((m, k), dtype=np.uint8)
    q[:, 0] = 0x38  # 1
    w = np.zeros((n, k), dtype=np.uint8)
    w[:, 0] = np.where(np.arange(n) % 2, 0xeb, 0xea)  # -88 and -80
    u = np.zeros((n, k), dtype=np.uint8)
    u[:, 0] = 0x38
    X = matrix(cuda_device, q, np.full((m, 2), 127, dtype=np.uint8), 1)
    G = matrix(cuda_device, w, np.full((2, 2), 127, dtype=np.uint8), 128)
    U = matrix(cuda_device, u, np.full((2, 2), 227, dtype=np.uint8), 128)
    g = F.values(w, np.full((2, 2), 127, dtype=np.uint8), 128)[:, 0]
    ref = np.tile(F.swiglu(g, 2.0 ** 100), (m, 1))
    # a subnormal reciprocal of 2^-127 or so is off by 2^-150 at most, the exponential by 2 + 1.2 * 88 units of 2^-23
    off = np.abs(ref) * (120 * 2.0 ** -23 + 2.0 ** -22)
    h, y = lib.bgq_f8_swiglu(G, U, X, want_out=True)
    assert (np.abs(f64(y) - ref) <= off + (np.abs(ref) + off) * 2.0 ** -8).all()
    check_codes(h, ref, off)
