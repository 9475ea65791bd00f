"""The e4m3 operators without a GPU: the oracle by hand, what the C entry points and the binding refuse."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import f8_oracle as F

FAKE = 0x10000000  # 256-byte aligned, never dereferenced: validation fails first
OUT, OTHER = FAKE + (1 << 20), FAKE + (2 << 20)  # results and a second result, which may not be an input


@pytest.fixture(scope="module")
def lib():
    from bit_group_quantized_gb300 import build, lib as L

    build.build()
    return L


# --------------------------------------------------------------------- oracle
def test_codes_by_hand():
    v = F.code_values()
    for code, value in {0x00: 0.0, 0x01: 2.0 ** -9, 0x07: 7 * 2.0 ** -9, 0x08: 2.0 ** -6, 0x38: 1.0, 0x3c: 1.5, 0x77: 240.0, 0x7e: 448.0,
                        0xb8: -1.0, 0x81: -(2.0 ** -9)}.items():
        assert v[code] == value
    assert math.isnan(v[0x7f]) and math.isnan(v[0xff])
    assert np.array_equal(v, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_rounding_by_hand():
    x = np.array([1.0625, 1.0624, 1.0626, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 440.0, 448.0, 432.0, 0.0])
    want = [0x38, 0x38, 0x39, 0x3a, 0xb8, 0x00, 0x02, 0x7e, 0x7e, 0x7e, 0x00]  # halves: to the even code
    assert F.nearest_codes(x).tolist() == want
    r = np.random.default_rng(1).standard_normal(5000) * 50
    assert np.array_equal(F.nearest_codes(r), torch.from_numpy(r).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scales_by_hand():
    assert F.scale_byte(448.0) == 127 and F.scale_byte(448.1) == 128 and F.scale_byte(224.0) == 126 and F.scale_byte(1.75) == 119
    assert F.scale_byte(0.0) == 0 and F.scale_byte(2.0 ** -140) == 0 and F.scale_byte(3.3e38) == 247
    q, s = F.quantise(np.array([[448.0] * 128 + [1.0] * 16, [0.0] * 128 + [np.inf] + [1.0] * 15]))
    assert s.tolist() == [[127, 119], [0, 127]]
    assert q[0].tolist() == [0x7e] * 128 + [0x78] * 16 and q[1].tolist() == [0] * 128 + [0x7f] * 16
    q, s = F.quantise(np.full((130, 16), 1.75) * np.arange(130)[:, None], 128)
    assert s.shape == (2, 1) and s[0, 0] == F.scale_byte(1.75 * 127) and s[1, 0] == F.scale_byte(1.75 * 129)


def test_values_take_their_block():
    q = np.full((129, 144), 0x38, dtype=np.uint8)
    v = F.values(q, np.array([[127, 128], [129, 130]], dtype=np.uint8), 128)
    assert v[127, 127] == 1 and v[127, 128] == 2 and v[128, 127] == 4 and v[128, 128] == 8
    h, a = F.norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(a, np.array([[3, 8]]) / math.sqrt(12.5))
    y, size = F.product(np.array([[1.0, -2.0]]), np.array([[3.0, 4.0]]))
    assert y.item() == -5 and size.item() == 11
    assert F.swiglu(0.0, 5.0) == 0 and abs(F.swiglu(40.0, 2.0) - 80) < 1e-12


# ------------------------------------------------------------------- refusals
def mat(lib, **kw):
    a = dict(q=FAKE, scale=FAKE, q_stride=256, scale_stride=4, rows=130, cols=256, block_rows=1)
    return lib.bgq_f8matrix(*{**a, **kw}.values())


BAD = [dict(q=None), dict(scale=None), dict(q=FAKE + 8), dict(scale=FAKE + 2), dict(rows=-1), dict(cols=0), dict(cols=264), dict(cols=-16),
       dict(q_stride=240), dict(q_stride=264), dict(scale_stride=0), dict(scale_stride=6), dict(cols=512 + 16, q_stride=1024), dict(block_rows=0),
       dict(block_rows=64)]
BIG = [dict(cols=65552, q_stride=65552, scale_stride=1024), dict(rows=1 << 24), dict(q_stride=1 << 36), dict(scale_stride=1 << 36)]


def calls(lib, matrix, **kw):
    """Each entry point on these matrices, the other arguments as they should be unless kw says otherwise."""
    L = lib.load()
    w = dict(block_rows=128)
    x, h, b, c = mat(lib), mat(lib, q=OUT, scale=OUT, cols=128), mat(lib, rows=128, **w), mat(lib, rows=128, **w)

    def ref(m):
        return None if m is False else C.byref(m)

    def quantise(m=matrix):
        k = {**dict(x=FAKE, xs=256), **kw}
        return L.bgq_f8_quantise(k["x"], k["xs"], ref(m), None)

    def norm(m=matrix):
        k = {**dict(h=OUT, delta=FAKE, f32=0, rho=FAKE, batch=130, d=256, eps=1e-6, a=OTHER), **kw}
        return L.bgq_rmsnorm_f8(k["h"], k["delta"], k["f32"], k["rho"], k["batch"], k["d"], k["eps"], ref(m), k["a"], None)

    def gemm(W=b, X=x):
        k = {**dict(y=OUT, yf=OTHER, ys=128, ws=FAKE, wsb=256), **kw}
        return L.bgq_f8_gemm(ref(W), ref(X), k["y"], k["yf"], k["ys"], k["ws"], k["wsb"], None)

    def swiglu(G=b, U=c, X=x, H=h):
        k = {**dict(y=OTHER, ys=128, ws=FAKE, wsb=256), **kw}
        return L.bgq_f8_swiglu(ref(G), ref(U), ref(X), ref(H), k["y"], k["ys"], k["ws"], k["wsb"], None)

    return quantise, norm, gemm, swiglu


def test_matrices_that_are_refused(lib):
    w = dict(block_rows=128)
    for bad, status in [(k, lib.ERR_INVALID_ARG) for k in BAD] + [(k, lib.ERR_UNSUPPORTED) for k in BIG]:
        m = mat(lib, **bad)
        quantise, norm, gemm, swiglu = calls(lib, m)
        assert quantise() == status, bad
        assert calls(lib, m, d=m.cols, batch=m.rows)[1]() == status, bad
        assert gemm(X=m) == status and gemm(W=mat(lib, **{**w, **bad})) == status, bad
        big = mat(lib, **{**w, **bad})
        assert swiglu(X=m) == status and swiglu(H=m) == status and swiglu(G=big) == status and swiglu(U=big) == status, bad
    quantise, norm, gemm, swiglu = calls(lib, False)
    assert quantise() == norm() == gemm(W=False) == gemm(X=False) == lib.ERR_INVALID_ARG
    assert swiglu(G=False) == swiglu(U=False) == swiglu(X=False) == lib.ERR_INVALID_ARG
    # inputs have a scale for each row, weights for 128 rows
    one, many = mat(lib), mat(lib, rows=128, **w)
    assert calls(lib, many)[1]() == gemm(W=mat(lib, rows=128)) == gemm(X=many) == swiglu(G=mat(lib, rows=128)) == lib.ERR_INVALID_ARG
    assert swiglu(U=mat(lib, rows=128)) == swiglu(X=many) == swiglu(H=mat(lib, cols=128, **w)) == lib.ERR_INVALID_ARG
    # shapes that do not fit each other
    assert gemm(W=mat(lib, rows=128, cols=240, **w)) == gemm(W=mat(lib, rows=0, **w)) == lib.ERR_INVALID_ARG
    assert swiglu(U=mat(lib, rows=144, **w)) == swiglu(H=mat(lib)) == swiglu(H=mat(lib, rows=129, cols=128)) == lib.ERR_INVALID_ARG
    odd = mat(lib, rows=120, **w)
    assert swiglu(G=odd, U=odd, H=False) == lib.ERR_INVALID_ARG  # 120 is no multiple of 16
    assert gemm(W=mat(lib, rows=(1 << 20) + 1, **w)) == lib.ERR_UNSUPPORTED
    assert one.rows == 130


def test_other_arguments_that_are_refused(lib):
    for kw in [dict(x=None), dict(x=FAKE + 8), dict(xs=248), dict(xs=260)]:
        assert calls(lib, mat(lib), **kw)[0]() == lib.ERR_INVALID_ARG, kw
    assert calls(lib, mat(lib), xs=1 << 36)[0]() == lib.ERR_UNSUPPORTED
    for kw in [dict(h=None), dict(h=FAKE + 8), dict(delta=FAKE + 4), dict(rho=FAKE + 2), dict(a=FAKE + 8), dict(batch=129), dict(batch=-1), dict(d=128),
               dict(eps=-1.0), dict(eps=math.nan)]:
        assert calls(lib, mat(lib), **kw)[1]() == lib.ERR_INVALID_ARG, kw
    for kw in [dict(y=None, yf=None), dict(y=FAKE + 8), dict(yf=FAKE + 4), dict(ys=120), dict(ys=132)]:
        assert calls(lib, mat(lib), **kw)[2]() == lib.ERR_INVALID_ARG, kw
    for kw in [dict(y=FAKE + 8), dict(ys=120), dict(ys=132)]:
        assert calls(lib, mat(lib), **kw)[3]() == lib.ERR_INVALID_ARG, kw
    assert calls(lib, mat(lib), y=None)[3](H=False) == lib.ERR_INVALID_ARG
    for kw in [dict(ws=None), dict(ws=FAKE + 16), dict(wsb=255)]:
        assert calls(lib, mat(lib), **kw)[2]() == calls(lib, mat(lib), **kw)[3]() == lib.ERR_WORKSPACE, kw
    L = lib.load()
    W, x = mat(lib, block_rows=128), mat(lib)
    assert L.bgq_f8_gemm_workspace_bytes(C.byref(W), C.byref(x)) == 256
    assert L.bgq_f8_gemm_workspace_bytes(C.byref(x), C.byref(x)) == 0


def test_results_over_inputs_are_refused(lib):
    m = mat(lib)
    for kw in [dict(h=FAKE), dict(a=OUT), dict(h=FAKE, delta=None)]:
        assert calls(lib, m, **kw)[1]() == lib.ERR_INVALID_ARG, kw
    assert calls(lib, m, y=FAKE)[2]() == calls(lib, m, yf=FAKE)[2]() == calls(lib, m, y=FAKE)[3]() == lib.ERR_INVALID_ARG
    square = mat(lib, cols=128, q=FAKE + (3 << 20))
    for h in (mat(lib, cols=128), mat(lib, cols=128, q=OUT), mat(lib, cols=128, scale=OUT)):
        assert calls(lib, m)[3](H=h) == lib.ERR_INVALID_ARG
    assert square.cols == 128


def test_nothing_to_do(lib):
    none, gone = mat(lib, rows=0), mat(lib, rows=0, q=OUT, scale=OUT, cols=128)
    assert calls(lib, none)[0]() == calls(lib, none, batch=0)[1]() == calls(lib, none)[2](X=none) == lib.OK
    assert calls(lib, none)[3](X=none, H=gone) == lib.OK


def test_binding_refuses_host_tensors(lib):
    q, s = torch.zeros(2, 128, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(2, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    for call in (lambda: lib.F8Matrix(q, s[:, :1]), lambda: lib.bgq_f8_quantise(torch.zeros(2, 128, dtype=torch.bfloat16)),
                 lambda: lib.bgq_rmsnorm_f8(torch.zeros(2, 128), None, 1e-6), lambda: lib.bgq_f8_gemm(None, None),
                 lambda: lib.bgq_f8_swiglu(None, None, None)):
        with pytest.raises(lib.BGQError) as e:
            call()
        assert e.value.status == lib.ERR_INVALID_ARG
