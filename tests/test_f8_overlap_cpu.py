"""Results of the e4m3 calls that share bytes with what the same call reads or writes are refused, wherever in each other they lie."""

import ctypes as C

import pytest

BASE = 0x10000000  # never dereferenced: the calls are refused
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from bit_group_quantized_gb300 import build, lib as L

    build.build()
    return L


def mat(lib, q, scale, rows=64, cols=256, block_rows=1, q_stride=256, scale_stride=4):
    return lib.bgq_f8matrix(q, scale, q_stride, scale_stride, rows, cols, block_rows)


def quantise(lib, m, x=BASE + 8 * MB, xs=256):
    return lib.load().bgq_f8_quantise(x, xs, C.byref(m), None)


def norm(lib, m, h=BASE + 8 * MB, delta=BASE + 9 * MB, f32=0, rho=BASE + 10 * MB, a=BASE + 11 * MB):
    return lib.load().bgq_rmsnorm_f8(h, delta, f32, rho, m.rows, m.cols, 1e-6, C.byref(m), a, None)


def gemm(lib, W, x, y=BASE + 8 * MB, yf=BASE + 9 * MB, ys=256):
    return lib.load().bgq_f8_gemm(C.byref(W), C.byref(x), y, yf, ys, BASE + 15 * MB, 256, None)


def swiglu(lib, g, u, x, h, y=BASE + 8 * MB, ys=256):
    return lib.load().bgq_f8_swiglu(C.byref(g), C.byref(u), C.byref(x), C.byref(h) if h else None, y, ys, BASE + 15 * MB, 256, None)


def test_quantiser(lib):
    bad = lib.ERR_INVALID_ARG
    x = BASE + 8 * MB  # 64 rows of 512 bytes
    for q in (x, x + 256, x + 63 * 512, x + 63 * 512 + 496, x - 63 * 256):
        assert quantise(lib, mat(lib, q, BASE)) == bad, q - x
    for s in (x, x + 1000, x + 64 * 512 - 4, x - 63 * 4):
        assert quantise(lib, mat(lib, BASE, s)) == bad, s - x
    for s in (BASE, BASE + 64 * 256 - 4):  # scales among the codes
        assert quantise(lib, mat(lib, BASE, s)) == bad
    # the rows of both in one buffer, 1024 bytes apart: codes over the values' end
    assert quantise(lib, mat(lib, x + 496, BASE, q_stride=1024), xs=512) == bad
    assert quantise(lib, mat(lib, x + 1024 - 240, BASE, q_stride=1024), xs=512) == bad


def test_norm(lib):
    bad = lib.ERR_INVALID_ARG
    h, delta, rho, a = (BASE + i * MB for i in (8, 9, 10, 11))
    m = mat(lib, BASE, BASE + MB)
    for kw in [dict(delta=h), dict(delta=h + 16), dict(delta=h + 64 * 1024 - 16), dict(a=h + 512), dict(a=delta), dict(a=delta + 4096),
               dict(rho=h + 1024), dict(rho=a), dict(rho=BASE), dict(delta=BASE + 16), dict(a=BASE + 256), dict(a=BASE + MB - 64 * 512 + 16),
               dict(delta=BASE + MB - 64 * 1024 + 16, f32=1), dict(h=BASE - 64 * 1024 + 16, delta=None), dict(h=a - 16, delta=None)]:
        assert norm(lib, m, **kw) == bad, kw
    for q in (h, h + 16, delta, delta + 64 * 512 - 16, a, rho):
        assert norm(lib, mat(lib, q, BASE + MB)) == bad
    for s in (h + 4, delta, a + 64 * 512 - 4, rho, BASE + 256):
        assert norm(lib, mat(lib, BASE, s)) == bad


def test_product(lib):
    bad = lib.ERR_INVALID_ARG
    W, x = mat(lib, BASE, BASE + MB, rows=256, block_rows=128), mat(lib, BASE + 2 * MB, BASE + 3 * MB)
    y = BASE + 8 * MB  # 64 rows of 512 bytes, 1024 in fp32
    for other in (BASE, BASE + 65536 - 16, BASE + MB, BASE + 2 * MB, BASE + 2 * MB + 16, BASE + 3 * MB, BASE + 3 * MB + 240):
        assert gemm(lib, W, x, y=other) == bad and gemm(lib, W, x, y=None, yf=other) == bad and gemm(lib, W, x, yf=other) == bad, other - BASE
    for yf in (y, y + 16, y + 64 * 512 - 16, y - 64 * 1024 + 16):
        assert gemm(lib, W, x, yf=yf) == bad
    # x's rows and results in one buffer, 512 bytes apart, 496 of them results
    assert gemm(lib, mat(lib, BASE, BASE + MB, rows=248, block_rows=128), mat(lib, y + 256, BASE + 3 * MB, q_stride=512), yf=None) == bad


def test_gated(lib):
    bad = lib.ERR_INVALID_ARG
    g, u = mat(lib, BASE, BASE + MB, rows=256, block_rows=128), mat(lib, BASE + 2 * MB, BASE + 3 * MB, rows=256, block_rows=128)
    x = mat(lib, BASE + 4 * MB, BASE + 5 * MB)
    y = BASE + 8 * MB
    good = mat(lib, BASE + 6 * MB, BASE + 7 * MB)
    for other in (BASE + 16, BASE + MB, BASE + 2 * MB + 256, BASE + 3 * MB, BASE + 4 * MB + 16, BASE + 5 * MB, BASE + 6 * MB + 16, BASE + 7 * MB + 16):
        assert swiglu(lib, g, u, x, good, y=other) == bad, other - BASE
        if other < BASE + 6 * MB:
            assert swiglu(lib, g, u, x, mat(lib, other, BASE + 7 * MB)) == bad and swiglu(lib, g, u, x, mat(lib, BASE + 6 * MB, other)) == bad
            assert swiglu(lib, g, u, x, mat(lib, other, BASE + 7 * MB), y=None) == bad
            assert swiglu(lib, g, u, x, None, y=other) == bad
    assert swiglu(lib, g, u, x, mat(lib, y, BASE + 7 * MB)) == swiglu(lib, g, u, x, mat(lib, BASE + 6 * MB, y + 64)) == bad
    assert swiglu(lib, g, u, x, mat(lib, BASE + 6 * MB, BASE + 6 * MB + 64), y=None) == bad
