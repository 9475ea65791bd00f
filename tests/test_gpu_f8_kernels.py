"""Each e4m3 product's kernel by name: the test asks the rule (csrc/f8_rule.h) that its size takes the kernel that it means.
Strides, neighbours, scales at the ends, NaN and rows far apart by the kernel for many rows, whose sizes lie further up than those of
the other tests of these; and long sums by all three.

The tolerances are those of test_gpu_f8.py, by its functions."""

import numpy as np
import pytest
import torch

import tests.test_gpu_f8 as one
import tests.test_gpu_f8_calls as calls
from bit_group_quantized_gb300 import lib
from oracle import f8_oracle as F
from tests.f8_rule import Choice
from tests.helpers import f64
from tests.test_gpu_f8 import U8, check_codes, matrix, random_matrix, sum_tolerance, swiglu_tolerance

pytestmark = pytest.mark.gpu

MANY = 20000  # rows that are many even for few rows of W and few columns
WIDER = 26000


def choice(m, n, k, gated=False):
    return Choice(m, n, k, gated, torch.cuda.get_device_properties(0).multi_processor_count)


def takes(name, m, n, k, gated=False):
    assert choice(m, n, k, gated).kernel == name, (m, n, k, gated)


# ------------------------------------------- what is tested of the others, by the kernel for many rows
def test_rows_apart(cuda_device):
    pads = dict(q_pad=48, s_pad=4)
    takes("many", MANY, 200, 656)
    one.check_gemm(cuda_device, MANY, 200, 656, pads=pads)
    takes("many", MANY, 208, 656, True)
    one.check_swiglu(cuda_device, MANY, 208, 656, pads=pads)


def test_narrower_tiles_rows_apart(cuda_device):
    takes("many", MANY, 150, 400)
    assert choice(MANY, 150, 400).wide < 256
    one.check_gemm(cuda_device, MANY, 150, 400, pads=dict(q_pad=80, s_pad=8))


@pytest.mark.parametrize("ex,ew", [(0, 254), (254, 0), (7, 247), (127, 127), (20, 120), (200, 150), (1, 160)])
def test_scales_at_the_ends(cuda_device, ex, ew):
    m, n, k = MANY, 130, 256
    takes("many", m, n, k)
    X = matrix(cuda_device, np.full((m, k), 0x38, dtype=np.uint8), np.full((m, 2), ex, dtype=np.uint8), 1)
    W = matrix(cuda_device, np.full((n, k), 0x38, dtype=np.uint8), np.full((2, 2), ew, dtype=np.uint8), 128)
    y = lib.bgq_f8_gemm(W, X, want_out=False, want_f32=True)[1]
    assert (f64(y) == k * 2.0 ** (ex + ew - 254)).all()


def test_nan_stays_in_its_row(cuda_device):
    takes("many", MANY, 150, 400)
    one.test_gemm_nan_stays_in_its_row(cuda_device, MANY)


def test_writes_its_rows_alone(cuda_device):
    takes("many", MANY, 133, 272)
    one.test_gemm_writes_its_rows_alone(cuda_device, MANY)
    takes("many", MANY, 144, 272, True)
    one.test_swiglu_writes_its_rows_alone(cuda_device, MANY)


# columns that end inside a TMA store's 16 bytes, at their end, inside a store and at its end, with whole tiles and narrower ones
@pytest.mark.parametrize("m,n,k,whole", [(5000, 1111, 272, True), (5000, 1112, 272, True), (5000, 1152, 272, True), (5003, 1028, 272, True),
                                         (2600, 2065, 528, False), (2601, 2072, 528, False), (2600, 2080, 528, False)])
def test_neighbours_of_results(cuda_device, m, n, k, whole):
    takes("many", m, n, k)
    assert (choice(m, n, k).wide == 256) == whole
    rng = np.random.default_rng(m + n)
    W, w = random_matrix(cuda_device, rng, n, k, 128)
    X, x = random_matrix(cuda_device, rng, m, k, 1)
    pitch = -(-n // 8) * 8 + 8
    wide = torch.full((m + 2, pitch), -7.0, dtype=torch.bfloat16, device=cuda_device)
    widef = torch.full((m + 2, pitch), -7.0, device=cuda_device)
    lib.bgq_f8_gemm(W, X, out=wide[1:m + 1, :n], out_f32=widef[1:m + 1, :n])
    ref, size = F.product(x, w)
    assert (np.abs(f64(widef[1:m + 1, :n]) - ref) <= sum_tolerance(size, k)).all()
    assert torch.equal(wide[1:m + 1, :n], widef[1:m + 1, :n].bfloat16())
    for t in (wide, widef):
        assert (t[:, n:] == -7).all() and (t[0] == -7).all() and (t[m + 1] == -7).all()


def test_blocks_that_are_not_finite(cuda_device):
    takes("many", WIDER, 272, 128, True)
    one.test_swiglu_blocks_that_are_not_finite(cuda_device, WIDER)


def test_far_negative_gates(cuda_device):
    takes("many", WIDER, 144, 256, True)
    one.test_swiglu_of_far_negative_gates(cuda_device, WIDER)


def test_rows_beyond_32_bits(cuda_device):
    takes("many", MANY, 144, 272)
    takes("many", MANY, 144, 272, True)
    calls.test_rows_beyond_32_bits(cuda_device, MANY)


def test_the_calls_tests_take_each_kernel():
    """The sizes of captured, shared and repeated calls: gated steps by each of the kernels."""
    assert [choice(m, n, k, True).kernel for m, n, k in calls.SHAPES] == ["few", "mid", "many"]
    assert [choice(m, n, k).kernel for m, n, k in calls.SHAPES] == ["few", "mid", "many"]


# ------------------------------------------------------------------ long sums
def gpu_values(m):
    """values(m) on the GPU, in 64 bits."""
    table = torch.from_numpy(F.code_values()).to(m.q.device)
    s = torch.exp2(m.scale.view(U8).double() - 127).repeat_interleave(m.block_rows, 0)[:m.rows].repeat_interleave(128, 1)[:, :m.cols]
    return table[m.q.view(U8).int()] * s


def product(x, w):
    return (x @ w.T).cpu().numpy(), (x.abs() @ w.abs().T).cpu().numpy()


def some(dev, gen, rows, cols, block, lo, hi):
    q = torch.randint(0, 127, (rows, cols), dtype=U8, device=dev, generator=gen) | torch.randint(0, 2, (rows, cols), dtype=U8, device=dev, generator=gen) << 7
    m = lib.F8Matrix.empty(rows, cols, block, dev)
    m.q.view(U8).copy_(q)
    m.scale.view(U8).copy_(torch.randint(lo, hi, m.scale.shape, dtype=U8, device=dev, generator=gen))
    return m


LONG = [("few", 3, 500, 8192), ("mid", 1, 70, 16384), ("mid", 40, 130, 65536), ("mid", 300, 300, 28688), ("mid", 1, 16, 65536),
        ("many", 1300, 1300, 16384), ("many", 1301, 1296, 65536), ("many", 1600, 1600, 13840)]


@pytest.mark.parametrize("name,m,n,k", LONG)
def test_long_sums(cuda_device, name, m, n, k):
    takes(name, m, n, k)
    gen = torch.Generator(device=cuda_device).manual_seed(m + n + k)
    W, X = some(cuda_device, gen, n, k, 128, 124, 131), some(cuda_device, gen, m, k, 1, 124, 131)
    y, yf = lib.bgq_f8_gemm(W, X, want_f32=True)
    ref, size = product(gpu_values(X), gpu_values(W))
    assert (np.abs(f64(yf) - ref) <= sum_tolerance(size, k)).all(), np.max(np.abs(f64(yf) - ref) / size)
    assert torch.equal(y, yf.bfloat16())


@pytest.mark.parametrize("name,m,n,k", [("few", 3, 512, 5120), ("mid", 1, 64, 16384), ("mid", 40, 144, 65536), ("many", 1100, 1104, 16384), ("many", 1040, 1040, 65536)])
def test_long_sums_gated(cuda_device, name, m, n, k):
    takes(name, m, n, k, True)
    gen = torch.Generator(device=cuda_device).manual_seed(m + n + k)
    lo = 122 - int(np.log2(k) / 2)  # gates of a few units
    G, U, X = (some(cuda_device, gen, *a) for a in ((n, k, 128, lo - 3, lo), (n, k, 128, lo - 1, lo + 2), (m, k, 1, 119, 122)))
    x = gpu_values(X)
    (g, sg), (u, su) = product(x, gpu_values(G)), product(x, gpu_values(U))
    ref, off = F.swiglu(g, u), swiglu_tolerance(g, u, sg, su, k)
    h, y = lib.bgq_f8_swiglu(G, U, X, want_out=True)
    assert (np.abs(f64(y) - ref) <= off + (np.abs(ref) + off) * 2.0 ** -8 + 2.0 ** -134).all()
    check_codes(h, ref, off)


@pytest.mark.parametrize("name,m,n,k", [("few", 3, 500, 8192), ("mid", 40, 130, 65536), ("many", 1300, 1300, 65536)])
def test_long_sums_of_one_sign(cuda_device, name, m, n, k):
    """All terms positive: a step's cut is then always downwards, and a sum is low by K / 32 units of 2^-23 at most, and never high by
    more than the additions of parts."""
    takes(name, m, n, k)
    gen = torch.Generator(device=cuda_device).manual_seed(k)
    W, X = some(cuda_device, gen, n, k, 128, 124, 131), some(cuda_device, gen, m, k, 1, 124, 131)
    W.q.view(U8).bitwise_and_(0x7f)
    X.q.view(U8).bitwise_and_(0x7f)
    ref, _ = product(gpu_values(X), gpu_values(W))
    off = (f64(lib.bgq_f8_gemm(W, X, want_out=False, want_f32=True)[1]) - ref) / ref
    assert off.min() >= -(k / 32 + 16) * 2.0 ** -23 and off.max() <= (k / 128 / 8 + 16) * 2.0 ** -23, (off.min(), off.max())
