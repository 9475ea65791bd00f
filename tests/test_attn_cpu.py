"""Attention operators without a GPU: the oracle's pins, the rotary plan against its definition, and every refusal
(argument checks come before any CUDA call)."""

import ctypes as C
import math

import numpy as np
import pytest

from oracle import attn_oracle as A
from oracle import bgq_oracle as O

FAKE = 0x10000000  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from bit_group_quantized_gb300 import build, lib as L

    build.build()
    return L


# ------------------------------------------------------------------ oracle pins
def test_rope_oracle_quarter_turn():
    # theta 1: every pair turns by its axis's position; two axes, two pairs each, columns (i, i + 4)
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y = A.rope(x, [[math.pi / 2], [math.pi]], 8, 1.0, [2, 2])
    assert np.allclose(y[0, 0], [-5, -6, -3, -4, 1, 2, -7, -8])
    y = A.rope(x, [[math.pi / 2], [math.pi]], 8, 1.0, [2, 2], pairs=True)
    assert np.allclose(y[0, 0], [-2, 1, -4, 3, -5, -6, -7, -8])
    assert np.allclose(A.rope(y, [[math.pi / 2], [math.pi]], 8, 1.0, [2, 2], pairs=True, inverse=True), x)


def test_rope_oracle_axes():
    assert A.rope_axes(6, [2, 2, 2]) == [0, 0, 1, 1, 2, 2]
    assert A.rope_axes(8, [4, 2, 2], cycle=True) == [0, 1, 2, 0, 1, 2, 0, 0]


def test_quantise_oracle_by_hand():
    x = np.zeros((1, 64))
    x[0, :4] = [-1.0, 14.0, 0.25, 0.5]  # scale 1, bias -1: codes 0, 15, floor(1.75), floor(2.0)
    code, scale, bias, _ = A.kv4_quantise(x)
    assert scale[0, 0] == 1.0 and bias[0, 0] == -1.0
    assert code[0, :5].tolist() == [0, 15, 1, 2, 1]
    sb = np.stack([O.f64_to_bf16_bits(scale), O.f64_to_bf16_bits(bias)], -1)
    assert A.kv4_values(A.kv4_pack(code), sb)[0, :4].tolist() == [-1.0, 14.0, 0.0, 1.0]


def test_quantise_oracle_constant_group():
    code, scale, bias, _ = A.kv4_quantise(np.full((2, 128), 3.5))
    assert not code.any() and not scale.any() and (bias == 3.5).all()


def test_attention_oracle_uniform_and_empty():
    # keys of zero: the mean of the values a row sees; a row before the first token sees none
    k_q, v_q = np.zeros((1, 1, 16, 8), np.uint32), np.zeros((1, 1, 16, 8), np.uint32)
    k_sb = np.zeros((1, 1, 16, 1, 2), np.uint16)
    v_sb = k_sb.copy()
    v_sb[0, 0, :, 0, 1] = O.f64_to_bf16_bits(np.arange(16.0))
    out, lse, _, _ = A.kv4_attention((k_q, k_sb, v_q, v_sb), [3], [0, 4], 5, None, np.ones((5, 2, 64)), 1.0)
    assert np.allclose(out[:, 0, 0], [0, 0, 0.5, 1, np.nan], equal_nan=True)
    assert np.allclose(lse[:4, 1], [-np.inf, 0, math.log(2), math.log(3)])
    out, _, _, _ = A.kv4_attention((k_q, k_sb, v_q, v_sb), [3], [0, 4], 4, None, np.ones((4, 1, 64)), 1.0, window=2)
    assert np.allclose(out[:, 0, 0], [0, 0, 0.5, 1.5])


# ------------------------------------------------------------------ rotary plan
def test_rope_plan_values(lib):
    p = lib.RopePlan(128, 64, 10000.0, [16, 8, 8]).c
    assert list(p.axis[:32]) == [0] * 16 + [1] * 8 + [2] * 8
    for i in range(32):
        want = 10000.0 ** (-i / 32) / (2 * math.pi)
        # two roundings of pow and the division (1e-15 relative), and the fixed point's last place, 2^-64 turns
        assert abs(p.freq[i] / 2.0 ** 64 - want) <= 1e-15 * want + 2.0 ** -64
    p = lib.RopePlan(64, 64, 100.0, [20, 6, 6], cycle=True).c
    assert list(p.axis[:32]) == A.rope_axes(32, [20, 6, 6], cycle=True)
    p = lib.RopePlan(64, 64, 100.0, [16, 16], restart=True).c
    assert p.freq[0] == p.freq[16] and p.freq[5] == p.freq[21]


@pytest.mark.parametrize("args", [(0, 64, 1e4, [32]), (128, 130, 1e4, [65]), (128, 64, 0.0, [32]), (128, 64, math.nan, [32]),
                                  (128, 64, math.inf, [32]), (128, 64, 1e4, []), (128, 64, 1e4, [16, 8]),
                                  (128, 64, 1e4, [40, -8])])
def test_rope_plan_invalid(lib, args):
    with pytest.raises(lib.BGQError) as e:
        lib.RopePlan(*args)
    assert e.value.status == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("args", [(512, 64, 1e4, [32]), (100, 64, 1e4, [32]), (128, 40, 1e4, [20]), (128, 64, 1e4, [4] * 8 + [0])])
def test_rope_plan_unsupported(lib, args):
    with pytest.raises(lib.BGQError) as e:
        lib.RopePlan(*args)
    assert e.value.status == lib.ERR_UNSUPPORTED


def test_rope_plan_flags(lib):
    p, sec = lib.bgq_rope_plan(), (C.c_int32 * 1)(32)
    L = lib.load()
    assert L.bgq_rope_init(C.byref(p), 64, 64, 1e4, 1, sec, 8) == lib.ERR_INVALID_ARG
    assert L.bgq_rope_init(C.byref(p), 64, 64, 1e4, 1, sec, 6) == lib.ERR_INVALID_ARG
    assert L.bgq_rope_init(None, 64, 64, 1e4, 1, sec, 0) == lib.ERR_INVALID_ARG
    assert L.bgq_rope_init(C.byref(p), 64, 64, 1e4, 1, None, 0) == lib.ERR_INVALID_ARG


# ------------------------------------------------------------------ refusals
def test_rope_refusals(lib):
    L = lib.load()
    plan = lib.RopePlan(128, 128, 1e4, [22, 21, 21])
    good = dict(p=plan.ref, x=FAKE, xs=512, pos=FAKE, ps=7, t=7, h=4, y=FAKE + 4096, ys=512, inv=0, st=None)
    bad = [dict(x=None), dict(x=FAKE + 2), dict(xs=504), dict(xs=516), dict(y=None), dict(y=FAKE + 8), dict(ys=511), dict(pos=None),
           dict(pos=FAKE + 2), dict(ps=6), dict(ps=-1), dict(t=-1), dict(h=0), dict(p=None), dict(y=FAKE, ys=520)]
    for b in bad:
        assert L.bgq_rope(*{**good, **b}.values()) == lib.ERR_INVALID_ARG, b
    assert L.bgq_rope(*{**good, **dict(h=1025, xs=1 << 20, ys=1 << 20)}.values()) == lib.ERR_UNSUPPORTED
    broken = lib.RopePlan(128, 128, 1e4, [64])
    broken.c.axis[3] = 1
    assert L.bgq_rope(*{**good, **dict(p=broken.ref)}.values()) == lib.ERR_INVALID_ARG
    assert L.bgq_rope(*{**good, **dict(t=0, ps=0)}.values()) == lib.OK  # nothing to do, nothing launched


def _cache(lib, **kw):
    a = dict(k_q=FAKE, k_sb=FAKE, v_q=FAKE, v_sb=FAKE, n_pages=4, page_size=16, kv_heads=2, head_dim=128)
    return lib.bgq_kv4_cache(*{**a, **kw}.values())


def _seqs(lib, **kw):
    a = dict(q_start=FAKE, kv_len=FAKE, pages=FAKE, batch=3, max_pages=2, rows=5, max_q=3)
    return lib.bgq_kv4_seqs(*{**a, **kw}.values())


BAD_CACHE = [dict(k_q=None), dict(k_sb=None), dict(v_q=None), dict(v_sb=None), dict(k_q=FAKE + 4), dict(v_sb=FAKE + 4),
             dict(n_pages=0), dict(page_size=8), dict(page_size=24), dict(kv_heads=0)]
BAD_SEQS = [dict(kv_len=None), dict(kv_len=FAKE + 2), dict(q_start=FAKE + 1), dict(pages=FAKE + 2), dict(batch=0),
            dict(rows=-1), dict(max_q=0), dict(max_pages=0), dict(q_start=None), dict(q_start=None, rows=3),
            dict(q_start=None, rows=4, max_q=1)]
BIG_CACHE = [dict(head_dim=96), dict(kv_heads=257)]


def _calls(lib, c, s):
    L = lib.load()
    return {"append": lambda **kw: L.bgq_kv4_append(C.byref(c), C.byref(s), *{**dict(k=FAKE, ks=256, v=FAKE, vs=256), **kw}.values(), None),
            "read": lambda **kw: L.bgq_kv4_read(C.byref(c), C.byref(s), *{**dict(k=FAKE, ks=256, v=FAKE, vs=256), **kw}.values(), None),
            "attention": lambda **kw: L.bgq_kv4_attention(
                C.byref(c), C.byref(s), *{**dict(q=FAKE, qs=1024, hq=8, scale=0.1, causal=1, window=0, out=FAKE, os=1024, lse=FAKE, ws=FAKE,
                                                 wsb=1 << 40), **kw}.values(), None)}


@pytest.mark.parametrize("which", ["append", "read", "attention"])
def test_kv4_refusals(lib, which):
    for kw in BAD_CACHE:
        assert _calls(lib, _cache(lib, **kw), _seqs(lib))[which]() == lib.ERR_INVALID_ARG, kw
    for kw in BAD_SEQS:
        assert _calls(lib, _cache(lib), _seqs(lib, **kw))[which]() == lib.ERR_INVALID_ARG, kw
    for kw in BIG_CACHE:
        assert _calls(lib, _cache(lib, **kw), _seqs(lib))[which]() == lib.ERR_UNSUPPORTED, kw
    assert _calls(lib, _cache(lib), _seqs(lib, batch=4097))[which]() == lib.ERR_UNSUPPORTED
    assert _calls(lib, _cache(lib), _seqs(lib, rows=0))[which]() == lib.OK  # nothing launched


@pytest.mark.parametrize("which", ["append", "read"])
def test_kv4_row_refusals(lib, which):
    call = _calls(lib, _cache(lib), _seqs(lib))[which]
    for kw in [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(ks=248), dict(ks=260), dict(vs=0), dict(vs=-256)]:
        assert call(**kw) == lib.ERR_INVALID_ARG, kw


def test_attention_refusals(lib):
    c, s = _cache(lib), _seqs(lib)
    call = _calls(lib, c, s)["attention"]
    for kw in [dict(q=None), dict(q=FAKE + 8), dict(qs=1016), dict(qs=1028), dict(out=None), dict(out=FAKE + 4), dict(os=8), dict(hq=0),
               dict(hq=7), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(lse=FAKE + 2)]:
        assert call(**kw) == lib.ERR_INVALID_ARG, kw
    assert call(hq=130, qs=1 << 16, os=1 << 16) == lib.ERR_UNSUPPORTED  # 65 query heads to a key head
    need = lib.load().bgq_kv4_attention_workspace_bytes(C.byref(c), C.byref(s), 8)
    assert need >= 256 and need % 256 == 0
    for kw in [dict(ws=None), dict(ws=FAKE + 16), dict(wsb=need - 1)]:
        assert call(**kw) == lib.ERR_WORKSPACE, kw
    assert lib.load().bgq_kv4_attention_workspace_bytes(C.byref(c), C.byref(s), 7) == 0


def test_binding_refuses_host_tensors(lib):
    import torch

    bf, i32 = torch.bfloat16, torch.int32
    with pytest.raises(lib.BGQError):
        lib.KV4Cache(*(torch.zeros(s, dtype=t) for _ in range(2) for s, t in (((1, 1, 16, 8), i32), ((1, 1, 16, 1, 2), bf))))
    with pytest.raises(lib.BGQError):
        lib.KV4Seqs(torch.zeros(1, dtype=i32))
    with pytest.raises(lib.BGQError):
        lib.bgq_rope(lib.RopePlan(64, 64, 1e4, [32]), torch.zeros(1, 1, 64, dtype=bf), torch.zeros(1, dtype=i32))


def test_counts_beyond_32_bits(lib):
    """What kernels would count past 2^31 is refused before anything is launched."""
    for kw in [dict(n_pages=2 ** 30, page_size=32), dict(n_pages=2 ** 31 - 1, kv_heads=2), dict(n_pages=2 ** 20, page_size=2 ** 16)]:
        for which in ("append", "read", "attention"):
            assert _calls(lib, _cache(lib, **kw), _seqs(lib))[which]() == lib.ERR_UNSUPPORTED, kw
    assert _calls(lib, _cache(lib, n_pages=2 ** 30 - 1), _seqs(lib, rows=0))["read"]() == lib.OK
    c, s = _cache(lib), _seqs(lib, rows=2 ** 30, max_q=2 ** 30)
    call = _calls(lib, c, s)["attention"]
    assert call(wsb=1 << 62) == lib.ERR_UNSUPPORTED  # 2^30 rows of 4 query heads to a key head
    s = _seqs(lib, rows=2 ** 29 - 2 ** 13, max_q=1)
    assert _calls(lib, c, s)["attention"](wsb=1 << 62) == lib.ERR_UNSUPPORTED  # rounded up to tiles it would pass 2^31


def test_attention_workspace_of_every_shape(lib):
    """Its size does not follow the lengths, and rows only where a unit of the list is kept for 128 or 256 of them."""
    size = lambda hq=8, **kw: lib.load().bgq_kv4_attention_workspace_bytes(  # noqa: E731
        C.byref(_cache(lib, head_dim=kw.pop("d", 128))), C.byref(_seqs(lib, **kw)), hq)
    for d in (64, 128, 256):
        one, many, most = size(d=d, q_start=None, rows=3, max_q=1), size(d=d, rows=1 << 12, max_q=1 << 12), size(d=d, rows=1 << 20, max_q=1 << 20)
        assert 4096 < one <= 16 << 20 and one < many <= 176 << 20
        assert many < most <= many + (1 << 20) * 4 // 128 * 64 + 4096
