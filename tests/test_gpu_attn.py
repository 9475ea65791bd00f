"""Attention operators on the GPU against the fp64 oracle: rotary positions, the 4-bit cache, attention over it, and a
decoder layer's attention block made of them.

Tolerances. A bf16 output is off by half a step, 2^-8 relative, beyond the kernel's own error. Attention's own error: the
kernels round the probabilities, and whole-prompt rows also the dequantised keys and values, to fp16 (2^-11 relative
each), so a score is off by at most 2^-11 * scale * sum|q k| =: e, a probability by 2e + 2^-10 relative, and an
output by (2e + 2^-10 + 2^-11) * sum p|v|. Few rows round p s (s the scale of v's group) instead, which multiplies
code - 8, while p (bias + 8 s) is summed in fp32: off by 2^-11 p s |code - 8| <= 2^-11 p 8 s, which does not shrink
where v itself is near zero, so A := sum p (|v| + 8 s) takes the place of sum p|v|. Sums in fp32 over at most some
thousand terms stay below 2^-12 of A, and of sum|q k| for a score: 2^-9 * (1 + scale * sum|q k|) * A covers all of them.
"""

import math

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib, synth
from oracle import attn_oracle as A
from oracle import bgq_oracle as O
from tests.helpers import bits16, f64, rel_l2

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32


def ints(v, dev):
    return torch.tensor(v, dtype=I32, device=dev)


def bf16(rng, *shape, dev, scale=1.0):
    return (torch.randn(*shape, generator=rng) * scale).to(BF).to(dev)


# ------------------------------------------------------------------ rotary positions
def rope_close(got, x, want, half, pairs):
    """2^-8 relative for the rounding, and for an angle off by 2^-21 (its fraction of a turn is exact to 2^-26 half
    turns, sincospi and the products add 2^-22) as much of the pair's length."""
    x = np.abs(x)
    length = np.zeros_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        length[..., a] = length[..., b] = np.hypot(x[..., a], x[..., b])
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * length).all()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens,heads,d,rot,sections", [(1, 1, 16, 16, [8]), (7, 5, 64, 32, [16]), (64, 40, 128, 128, [16, 24, 24]),
                                                         (33, 3, 96, 48, [10, 14]), (2500, 1, 256, 256, [128]), (5, 129, 256, 192, [32, 32, 32]),
                                                         (1300, 12, 64, 64, [1, 1, 30])])
def test_rope(cuda_device, tokens, heads, d, rot, sections, pairs):
    rng = torch.Generator().manual_seed(tokens)
    wide = bf16(rng, tokens, heads + 2, d, dev=cuda_device)
    x = wide[:, 1:1 + heads]
    pos = torch.randint(-1000, 1 << 20, (len(sections), tokens), generator=rng, dtype=I32)
    pos[:, -1] = 2 ** 31 - 1
    pos[-1, 0] = -2 ** 31
    plan = lib.RopePlan(d, rot, 10000.0, sections, pairs=pairs)
    for inverse in (False, True):
        y = lib.bgq_rope(plan, x, pos.to(cuda_device), inverse=inverse)
        want = A.rope(f64(x), pos.numpy(), rot, 10000.0, sections, pairs=pairs, inverse=inverse)
        rope_close(f64(y), f64(x), want, rot // 2, pairs)
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("kw", [dict(cycle=True), dict(restart=True), dict(restart=True, pairs=True)])
def test_rope_axes_layouts(cuda_device, kw):
    rng = torch.Generator().manual_seed(3)
    x = bf16(rng, 20, 4, 64, dev=cuda_device)
    pos = torch.randint(0, 5000, (3, 20), generator=rng, dtype=I32)
    y = lib.bgq_rope(lib.RopePlan(64, 64, 5000.0, [12, 10, 10], **kw), x, pos.to(cuda_device))
    want = A.rope(f64(x), pos.numpy(), 64, 5000.0, [12, 10, 10], **kw)
    rope_close(f64(y), f64(x), want, 32, kw.get("pairs", False))


def test_rope_in_place_beside_others(cuda_device):
    """The query and key heads of a fused projection turned where they stand; the value heads keep their bits."""
    rng = torch.Generator().manual_seed(4)
    qkv = bf16(rng, 50, 12, 128, dev=cuda_device)
    before = qkv.clone()
    pos = torch.arange(50, dtype=I32, device=cuda_device)
    plan = lib.RopePlan(128, 128, 10000.0, [64])
    want = lib.bgq_rope(plan, before[:, :10], pos)
    assert lib.bgq_rope(plan, qkv[:, :10], pos, y=qkv[:, :10]).data_ptr() == qkv.data_ptr()
    assert torch.equal(qkv[:, :10], want) and torch.equal(qkv[:, 10:], before[:, 10:])


def test_rope_gradient(cuda_device):
    """inverse is the transpose of the forward turn: <g, turn(x)> = <inverse(g), x> for every unit vector pair, here by
    random vectors, and by differences of the (linear) map along single columns."""
    rng = torch.Generator().manual_seed(5)
    plan = lib.RopePlan(64, 48, 10000.0, [10, 14])
    pos = torch.randint(0, 300, (2, 9), generator=rng, dtype=I32).to(cuda_device)
    x, g = bf16(rng, 9, 2, 64, dev=cuda_device), bf16(rng, 9, 2, 64, dev=cuda_device)
    gx = lib.bgq_rope(plan, g, pos, inverse=True)
    y = lib.bgq_rope(plan, x, pos)
    # each side is a sum of 1152 products whose bf16 factor is off by 2^-8 relative
    lhs, rhs = (f64(g) * f64(y)), (f64(gx) * f64(x))
    assert abs(lhs.sum() - rhs.sum()) <= 2.0 ** -8 * (np.abs(lhs).sum() + np.abs(rhs).sum())
    for col in (0, 5, 23, 24, 47, 50):
        e = torch.zeros_like(x)
        e[..., col] = 1.0
        d = f64(lib.bgq_rope(plan, e, pos))  # column col of the Jacobian, entries off by 2^-8 relative
        want = (f64(g) * d).sum(-1)
        tol = 2.0 ** -8 * (np.abs(f64(g) * d).sum(-1) + np.abs(want)) + 2.0 ** -21 * np.abs(f64(g)).sum(-1)
        assert (np.abs(f64(gx)[..., col] - want) <= tol).all()


# ------------------------------------------------------------------ the cache
class Case:
    """Sequences with their tokens already in a cache of randomly placed pages; their page lists have room for `room` tokens
    or more (those behind a sequence's own are -1)."""

    def __init__(self, dev, kv, new, hkv, d, page, seed=0, spare=2, pages=True, gap=0, behind=0, room=2048):
        rng = torch.Generator().manual_seed(seed)
        self.dev, self.kv, self.new, self.d, self.hkv = dev, kv, new, d, hkv
        B = len(kv)
        if pages:
            need = [max(-(-n // page), 0) for n in kv]
            self.n_pages = sum(need) + spare
            order = torch.randperm(self.n_pages, generator=rng).tolist()
            table = np.full((B, max(max(need), 1, -(-room // page))), -1, dtype=np.int32)
            for b, n in enumerate(need):
                for i in range(n):
                    table[b, i] = order.pop()
            self.pages = table
        else:
            page = max(16, -(-max(kv) // 16) * 16)
            self.n_pages, self.pages = B, None
        self.page = page
        self.q_start = [gap]
        for m in new:
            self.q_start.append(self.q_start[-1] + m)
        self.rows = self.q_start[-1] + behind
        col = torch.exp(0.4 * torch.randn(hkv, 1, d, generator=rng))
        k = (torch.randn(self.n_pages, hkv, page, d, generator=rng) * col).to(BF)
        v = torch.randn(self.n_pages, hkv, page, d, generator=rng).to(BF)
        self.np = []
        for x in (k, v):
            code, scale, bias, _ = A.kv4_quantise(f64(x))
            self.np += [A.kv4_pack(code).astype(np.uint32), np.stack([O.f64_to_bf16_bits(scale), O.f64_to_bf16_bits(bias)], -1)]
        self.rng = rng

    def cache(self):
        t = []
        for i, a in enumerate(self.np):
            t.append(torch.from_numpy(a.view(np.int32).copy()).to(self.dev) if i % 2 == 0
                     else torch.from_numpy(a.astype(np.uint16).view(np.int16).copy()).view(BF).to(self.dev))
        return lib.KV4Cache(*t)

    def seqs(self):
        table = None if self.pages is None else torch.from_numpy(self.pages).to(self.dev)
        return lib.KV4Seqs(ints(self.kv, self.dev), rows=self.rows, pages=table, q_start=ints(self.q_start, self.dev),
                           max_q=max(max(self.new), 1))

    def oracle(self, q, scale=None, causal=True, window=0):
        return A.kv4_attention(self.np, self.kv, self.q_start, self.rows, self.pages, f64(q), self.d ** -0.5 if scale is None else scale,
                               causal, window)


def slots(c: Case):
    """(page, place) of every row, None where it has none."""
    got = [None] * c.rows
    for b, (n, m) in enumerate(zip(c.kv, c.new)):
        for j in range(m):
            got[c.q_start[b] + j] = A.slot(max(n, 0) - m + j, b, c.pages, c.page, c.n_pages)
    return got


WRITES = [dict(kv=[1], new=[1], hkv=1, d=64, page=16), dict(kv=[17, 300, 5], new=[1, 1, 1], hkv=3, d=128, page=16),
          dict(kv=[40, 0, 70, 9], new=[40, 0, 33, 9], hkv=2, d=256, page=32), dict(kv=[1500, 700], new=[1500, 350], hkv=8, d=128, page=64),
          dict(kv=[3, 20], new=[5, 2], hkv=1, d=64, page=16), dict(kv=[33, 48], new=[33, 2], hkv=40, d=256, page=16, pages=False)]


@pytest.mark.parametrize("kw", WRITES)
def test_append_and_read(cuda_device, kw):
    c = Case(cuda_device, seed=1, gap=2, behind=3, **kw)
    wide = bf16(c.rng, c.rows, 2 * c.hkv + 1, c.d, dev=cuda_device)
    k, v = wide[:, :c.hkv], wide[:, c.hkv + 1:]  # two parts of one projection's rows
    k[c.rows // 2, 0] = 1.5  # a constant group
    cache, seqs = c.cache(), c.seqs()
    lib.bgq_kv4_append(cache, seqs, k, v)
    want = [a.copy() for a in c.np]
    where, edges = slots(c), 0
    for i, x in ((0, k), (2, v)):
        code, scale, bias, edge = A.kv4_quantise(f64(x))
        words, sb = A.kv4_pack(code), np.stack([O.f64_to_bf16_bits(scale), O.f64_to_bf16_bits(bias)], -1)
        edges += int((edge < 2.0 ** -17).sum())  # nearer to a half than fp32 tells apart: none in this data
        for r, at in enumerate(where):
            if at is not None:
                want[i][at[0], :, at[1]], want[i + 1][at[0], :, at[1]] = words[r], sb[r]
    assert edges == 0
    for t, w in zip((cache.k_q, cache.k_sb, cache.v_q, cache.v_sb), want):
        got = t.cpu().numpy().view(np.uint32) if t.dtype == I32 else bits16(t)
        assert np.array_equal(got, w.astype(got.dtype))
    # and back: rows of no sequence keep what they held
    ko, vo = (torch.full((c.rows, c.hkv, c.d), 7.0, dtype=BF, device=cuda_device) for _ in range(2))
    lib.bgq_kv4_read(cache, seqs, k=ko, v=vo)
    for o, i in ((ko, 0), (vo, 2)):
        for r, at in enumerate(where):
            got = f64(o[r])
            if r < c.q_start[0] or r >= c.q_start[-1]:
                assert (got == 7.0).all()
            elif at is None:
                assert (got == 0.0).all()
            else:
                val = A.kv4_values(want[i][at[0], :, at[1]], want[i + 1][at[0], :, at[1]])
                assert (np.abs(got - val) <= 2.0 ** -8 * np.abs(val) + 2.0 ** -22 * np.abs(val).max()).all()


def test_append_non_finite_groups(cuda_device):
    c = Case(cuda_device, [20], [4], 2, 128, 16)
    k, v = bf16(c.rng, 4, 2, 128, dev=cuda_device), bf16(c.rng, 4, 2, 128, dev=cuda_device)
    k[0, 0, 5], k[1, 1, 127], v[2, 0, 64], v[3, 1, 0] = math.nan, math.inf, -math.inf, math.nan
    k[2, 1, 3], k[2, 1, 4] = 3e38, -3e38  # finite, a range beyond fp32
    cache, seqs = c.cache(), c.seqs()
    lib.bgq_kv4_append(cache, seqs, k, v)
    ko, vo = lib.bgq_kv4_read(cache, seqs)
    nk, nv = torch.isnan(ko), torch.isnan(vo)
    want_k, want_v = torch.zeros_like(nk), torch.zeros_like(nv)
    want_k[0, 0, :64] = want_k[1, 1, 64:] = want_k[2, 1, :64] = True
    want_v[2, 0, 64:] = want_v[3, 1, :64] = True
    assert torch.equal(nk, want_k) and torch.equal(nv, want_v)


def test_absent_pages_are_passed_over(cuda_device):
    c = Case(cuda_device, [70, 40], [70, 40], 2, 64, 16, spare=0)
    c.pages[0, 1], c.pages[1, 0], c.pages[0, 3] = -1, c.n_pages, 2 ** 30
    before = [a.copy() for a in c.np]
    cache, seqs = c.cache(), c.seqs()
    k = bf16(c.rng, c.rows, 2, 64, dev=cuda_device)
    lib.bgq_kv4_append(cache, seqs, k, k)
    ko, vo = lib.bgq_kv4_read(cache, seqs)
    where = slots(c)
    touched = {at for at in where if at}
    for p in range(c.n_pages):
        for t in range(16):
            same = np.array_equal(cache.k_q[p, :, t].cpu().numpy().view(np.uint32), before[0][p, :, t])
            assert same == ((p, t) not in touched)
    for r, at in enumerate(where):
        assert bool((ko[r] == 0).all()) == (at is None) and bool((vo[r] == 0).all()) == (at is None)


# ------------------------------------------------------------------ attention
def attn_close(c, q, out, lse, scale=None, causal=True, window=0):
    o, l, a, s = c.oracle(q, scale, causal, window)
    live = ~np.isnan(l)
    got, gl = f64(out), f64(lse)
    tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -9 * (1 + s)[..., None] * a
    assert (np.abs(got - o) <= tol)[live].all(), np.nanmax((np.abs(got - o) / np.maximum(tol, 1e-30))[live])
    assert rel_l2(got[live], o[live]) <= 2.0 ** -8
    none = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl) & live, none)
    seen = live & ~none
    assert (np.abs(gl[seen] - l[seen]) <= 2.0 ** -10 * (s[seen] + 1)).all()
    assert (got[none] == 0).all()
    return live


ATTN = [
    dict(kv=[1], new=[1], hq=1, hkv=1, d=64, page=16), dict(kv=[513], new=[1], hq=32, hkv=8, d=128, page=64),
    dict(kv=[33, 0, 16, 700, 1], new=[1, 1, 1, 1, 1], hq=8, hkv=2, d=128, page=16),
    dict(kv=[1000], new=[1], hq=64, hkv=1, d=256, page=16), dict(kv=[257, 90], new=[1, 1], hq=6, hkv=2, d=256, page=48),
    dict(kv=[2000, 31], new=[1, 1], hq=4, hkv=4, d=64, page=128), dict(kv=[300, 64, 65, 20], new=[5, 3, 8, 0], hq=16, hkv=2, d=256, page=16),
    dict(kv=[130, 47], new=[6, 2], hq=9, hkv=3, d=64, page=32), dict(kv=[3, 40], new=[7, 40], hq=4, hkv=2, d=128, page=16),
    dict(kv=[200], new=[200], hq=8, hkv=2, d=128, page=64), dict(kv=[311, 150, 129], new=[150, 1, 129], hq=4, hkv=1, d=128, page=16),
    dict(kv=[160], new=[96], hq=10, hkv=2, d=64, page=32), dict(kv=[140, 260], new=[100, 33], hq=6, hkv=2, d=256, page=64),
    dict(kv=[90, 400], new=[1, 1], hq=8, hkv=8, d=128, page=16, pages=False), dict(kv=[270], new=[270], hq=3, hkv=1, d=128, page=16, pages=False),
]
MASKS = [(True, 0), (False, 0), (True, 7), (True, 100), (False, 64)]


@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("kw", ATTN)
def test_attention(cuda_device, kw, causal, window):
    kw = dict(kw)
    hq = kw.pop("hq")
    c = Case(cuda_device, seed=2, gap=1, behind=2, **kw)
    wide = bf16(c.rng, c.rows, hq + 1, c.d, dev=cuda_device, scale=1.5)
    q = wide[:, 1:]
    out = torch.full((c.rows, hq + 2, c.d), 7.0, dtype=BF, device=cuda_device)
    o = out[:, 1:-1]
    lse = torch.full((c.rows, hq), 7.0, device=cuda_device)
    lib.bgq_kv4_attention(c.cache(), c.seqs(), q, causal=causal, window=window, out=o, lse=lse)
    live = attn_close(c, q, o, lse, causal=causal, window=window)
    dead = torch.from_numpy(~live).to(cuda_device)
    assert (o[dead] == 7.0).all() and (lse[dead] == 7.0).all()  # rows of no sequence, and other heads, are left alone
    assert (out[:, 0] == 7.0).all() and (out[:, -1] == 7.0).all()
    assert dead.any()


@pytest.mark.parametrize("new", [1, 4, 120])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_masked_tokens_never_reach_a_row(cuda_device, d, new):
    """NaN and infinities in the slots behind the last token, in given-up pages, and in tokens that causality or the window hides: the
    same bits as with ordinary values there."""
    c = Case(cuda_device, [150, 129, 131], [new, min(new, 5), new], 2, d, 16)
    c.pages[1, 2] = -1
    q = bf16(c.rng, c.rows, 8, d, dev=cuda_device, scale=1.5)
    bad = np.array([0x7fc0, 0x7f80, 0xff80, 0x7fc0], dtype=np.uint16)
    outs = []
    for poison in (False, True):
        cache, seqs = c.cache(), c.seqs()
        if poison:
            held = {A.slot(t, b, c.pages, 16, c.n_pages) for b, n in enumerate(c.kv) for t in range(n)}
            # the last token of sequence 0 is hidden from all rows but its last, the first ones by the window
            hide = [A.slot(t, 0, c.pages, 16, c.n_pages) for t in list(range(0, 150 - new - 40)) + ([149] if new > 1 else [])]
            for p in range(c.n_pages):
                for t in range(16):
                    if (p, t) not in held or (p, t) in hide:
                        v = torch.from_numpy(np.roll(bad, t).view(np.int16).copy()).view(BF).to(cuda_device)
                        cache.k_sb[p, :, t, :, :] = v[0]
                        cache.v_sb[p, :, t, :, 0], cache.v_sb[p, :, t, :, 1] = v[1], v[2]
        out, lse = lib.bgq_kv4_attention(cache, seqs, q, window=41, want_lse=True)
        outs.append((out, lse))
    live = torch.ones(c.rows, dtype=torch.bool, device=cuda_device)
    if new > 1:
        live[new - 1] = False  # sequence 0's last row does see its poisoned token
        assert torch.isnan(outs[1][0][new - 1]).all()
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a[live], b[live])


def test_nan_reaches_the_rows_that_see_it(cuda_device):
    """A NaN group of a value reaches its 64 columns of the rows that see it, a NaN group of a key every column."""
    for d, new in ((64, 1), (128, 3), (128, 60), (256, 70)):
        c = Case(cuda_device, [100], [new], 1, d, 32)
        q = bf16(c.rng, c.rows, 2, d, dev=cuda_device)
        page, at = A.slot(97, 0, c.pages, 32, c.n_pages)
        row = torch.arange(new, device=cuda_device) + 100 - new >= 97  # by position
        cache = c.cache()
        clean, _ = lib.bgq_kv4_attention(cache, c.seqs(), q)
        cache.v_sb[page, 0, at, 0, :] = math.nan
        out, _ = lib.bgq_kv4_attention(cache, c.seqs(), q)
        bad = torch.isnan(out)
        assert bad[row][..., :64].all() and not bad[row][..., 64:].any() and not bad[~row].any()
        assert torch.equal(out[~row], clean[~row]) and torch.isfinite(clean).all()
        cache = c.cache()
        cache.k_sb[page, 0, at, d // 64 - 1, :] = math.nan
        out, lse = lib.bgq_kv4_attention(cache, c.seqs(), q, want_lse=True)
        assert torch.isnan(out[row]).all() and torch.isnan(lse[row]).all() and torch.equal(out[~row], clean[~row])


@pytest.mark.parametrize("new", [1, 90])
def test_nan_and_infinite_queries_stay_in_their_rows(cuda_device, new):
    c = Case(cuda_device, [100], [new], 2, 128, 32)
    q = bf16(c.rng, c.rows, 8, 128, dev=cuda_device)
    clean, _ = lib.bgq_kv4_attention(c.cache(), c.seqs(), q)
    q2 = q.clone()
    q2[0, 1, 7], q2[-1, 6, 100] = math.nan, math.inf
    out, _ = lib.bgq_kv4_attention(c.cache(), c.seqs(), q2)
    hit = torch.zeros(c.rows, 8, dtype=torch.bool, device=cuda_device)
    hit[0, 1] = hit[-1, 6] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("new", [1, 5, 64])
@pytest.mark.parametrize("kexp,vexp,qexp", [(0, 20, 0), (-20, -30, 20), (30, 90, -30), (100, -100, -100), (-60, 0, 60)])
def test_values_beyond_half_precision(cuda_device, kexp, vexp, qexp, new):
    """Keys, values and queries whose sizes leave fp16's range: powers of two carry through exactly."""
    c = Case(cuda_device, [140], [new], 2, 128, 16)
    q = bf16(c.rng, c.rows, 4, 128, dev=cuda_device)
    for i, e in ((1, kexp), (3, vexp)):
        c.np[i] = O.f64_to_bf16_bits(O.bf16_to_f64(c.np[i]) * 2.0 ** e)
    q = (q.double() * 2.0 ** qexp).to(BF)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    attn_close(c, q, out, lse)


@pytest.mark.parametrize("new", [1, 64])
def test_token_scales_of_different_sizes(cuda_device, new):
    """Tokens whose scales differ by 2^12 within a sequence, large ones first, last and in the middle."""
    for big in (0, 70, 139):
        c = Case(cuda_device, [140], [new], 1, 64, 16)
        for t in range(140):
            p, at = A.slot(t, 0, c.pages, 16, c.n_pages)
            if abs(t - big) < 3:
                c.np[3][p, :, at] = O.f64_to_bf16_bits(O.bf16_to_f64(c.np[3][p, :, at]) * 2.0 ** 12 * (1 if t % 2 else 2 ** 8))
        q = bf16(c.rng, c.rows, 3, 64, dev=cuda_device)
        out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
        attn_close(c, q, out, lse)


@pytest.mark.parametrize("new", [1, 70])
def test_peaked_and_flat_scores(cuda_device, new):
    """Scores of some hundreds (one token takes all) and all alike (scale 0: the mean)."""
    c = Case(cuda_device, [300], [new], 2, 128, 64)
    q = bf16(c.rng, c.rows, 4, 128, dev=cuda_device, scale=30.0)
    for scale in (0.0, 0.3, -0.3):
        out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, scale=scale, want_lse=True)
        o, l, a, s = c.oracle(q, scale)
        e = 2.0 ** -9 * (1 + s)  # a score's error is too large here for the linear bound: exp(2e) - 1 takes its place
        tol = 2.0 ** -8 * np.abs(o) + np.expm1(2 * e)[..., None] * a
        assert (np.abs(f64(out) - o) <= tol).all() and (np.abs(f64(lse) - l) <= e).all()


def test_lengths_grow_under_a_captured_graph(cuda_device):
    """rope, append and attention of a decode step captured once and replayed while the lengths on the device grow; two
    graphs with workspaces of their own replayed in turn give the bits of direct calls."""
    B, hq, hkv, d, page = 3, 8, 2, 128, 16
    c = Case(cuda_device, [30, 5, 47], [1, 1, 1], hkv, d, page, spare=9, room=0)
    table = np.full((B, 6), -1, dtype=np.int32)
    free = [p for p in range(c.n_pages) if p not in c.pages]
    table[:, :c.pages.shape[1]] = c.pages
    for b in range(B):
        for i in range(6):
            if table[b, i] < 0 and free and i * page < c.kv[b] + 8:
                table[b, i] = free.pop()
    plan = lib.RopePlan(d, d, 10000.0, [64])
    pages = torch.from_numpy(table).to(cuda_device)
    qkv = torch.empty(B, hq + 2 * hkv, d, dtype=BF, device=cuda_device)

    def state():
        s = dict(kv=ints(c.kv, cuda_device), pos=ints([n - 1 for n in c.kv], cuda_device), cache=c.cache(),
                 out=torch.empty(B, hq, d, dtype=BF, device=cuda_device), turned=torch.empty(B, hq + hkv, d, dtype=BF, device=cuda_device))
        s["seqs"] = lib.KV4Seqs(s["kv"], pages=pages)
        s["ws"] = lib.workspace(lib.kv4_attention_workspace_bytes(s["cache"], s["seqs"], hq), cuda_device)
        return s

    def step(s):
        lib.bgq_rope(plan, qkv[:, :hq + hkv], s["pos"], y=s["turned"])
        lib.bgq_kv4_append(s["cache"], s["seqs"], s["turned"][:, hq:], qkv[:, hq + hkv:])
        lib.bgq_kv4_attention(s["cache"], s["seqs"], s["turned"][:, :hq], out=s["out"], ws=s["ws"])

    direct, two = state(), [state(), state()]
    graphs = []
    for s in two:
        qkv.normal_()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(s)  # once before the capture
        torch.cuda.current_stream().wait_stream(side)
        for name, a in zip(("k_q", "k_sb", "v_q", "v_sb"), c.np):
            t = getattr(s["cache"], name)
            t.copy_(getattr(direct["cache"], name))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    rng = torch.Generator().manual_seed(8)
    for _ in range(6):
        qkv.copy_(bf16(rng, B, hq + 2 * hkv, d, dev="cpu"))
        for s in [direct] + two:
            s["kv"] += 1
            s["pos"] += 1
        step(direct)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s in two:
            assert torch.equal(s["out"], direct["out"]) and torch.equal(s["cache"].k_q, direct["cache"].k_q)


def test_other_stream_and_same_bits(cuda_device):
    c = Case(cuda_device, [2000, 900, 31], [1, 1, 1], 2, 128, 16)
    q = bf16(c.rng, 3, 16, 128, dev=cuda_device)
    cache, seqs = c.cache(), c.seqs()
    first, _ = lib.bgq_kv4_attention(cache, seqs, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, _ = lib.bgq_kv4_attention(cache, seqs, q, stream=side)
    ws = lib.workspace(lib.kv4_attention_workspace_bytes(cache, seqs, 16), cuda_device)
    again = [lib.bgq_kv4_attention(cache, seqs, q, ws=ws)[0] for _ in range(3)]  # a used workspace serves again
    torch.cuda.synchronize()
    for o in [other] + again:
        assert torch.equal(o, first)


def test_no_rows(cuda_device):
    c = Case(cuda_device, [20, 3], [0, 0], 1, 64, 16)
    q = torch.empty(0, 2, 64, dtype=BF, device=cuda_device)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    lib.bgq_kv4_append(c.cache(), c.seqs(), q[:, :1], q[:, :1])
    assert lib.bgq_kv4_read(c.cache(), c.seqs())[0].shape == (0, 1, 64)
    assert lib.bgq_rope(lib.RopePlan(64, 64, 1e4, [32]), q, torch.empty(0, dtype=I32, device=cuda_device)).shape == (0, 2, 64)


@pytest.mark.parametrize("new", [1, 70])
def test_offsets_past_32_bits(cuda_device, new):
    """Pages whose codes lie more than 2^32 bytes, and words, into a large pool: the bits of a small pool."""
    d, hkv, page = 128, 4, 64
    c = Case(cuda_device, [150], [new], hkv, d, page, spare=0)
    q = bf16(c.rng, c.rows, 8, d, dev=cuda_device)
    k = bf16(c.rng, c.rows, hkv, d, dev=cuda_device)
    small, seqs = c.cache(), c.seqs()
    lib.bgq_kv4_append(small, seqs, k, k)
    want, _ = lib.bgq_kv4_attention(small, seqs, q)
    n = (1 << 32) // (hkv * page * d // 8) + 8  # words
    big = lib.KV4Cache(*(torch.empty(s, dtype=t, device=cuda_device) for _ in range(2)
                         for s, t in (((n, hkv, page, d // 8), I32), ((n, hkv, page, d // 64, 2), BF))))
    old = c.cache()
    for name in ("k_q", "k_sb", "v_q", "v_sb"):
        getattr(big, name)[-c.n_pages:] = getattr(old, name)
    far = lib.KV4Seqs(seqs.kv_len, rows=c.rows, pages=seqs.pages + (n - c.n_pages), q_start=seqs.q_start, max_q=new)
    lib.bgq_kv4_append(big, far, k, k)
    got, _ = lib.bgq_kv4_attention(big, far, q)
    assert torch.equal(got, want)
    for a, b in zip(lib.bgq_kv4_read(big, far), lib.bgq_kv4_read(small, seqs)):
        assert torch.equal(a, b)


def test_attention_block_of_a_decoder_layer(cuda_device):
    """A decode step of a layer's attention block through the library alone: RMSNorm, the 4-bit query/key/value projection, rotary
    positions, the cache, attention over it, the 4-bit output projection with its residual."""
    B, dm, hq, hkv, d, page = 4, 1024, 8, 2, 128, 16
    kv = [37, 1, 130, 64]
    c = Case(cuda_device, kv, [1] * B, hkv, d, page)
    mats = []
    for i, (r, cols) in enumerate((((hq + 2 * hkv) * d, dm), (dm, hq * d))):
        q, sb = synth.qmatrix(20 + i, r, cols, 4)
        mats.append((q, sb, lib.QMatrix(q.to(cuda_device), sb.to(cuda_device), r, cols, 4)))
    rho = synth.rho(20, 0, dm)
    h = torch.randn(B, dm, generator=c.rng)
    a = lib.bgq_rmsnorm(h.to(cuda_device), rho.to(cuda_device), 1e-6)
    qkv = lib.q4_gemv(mats[0][2], a)
    qkv = (qkv.float() / qkv.float().std()).to(BF).view(B, hq + 2 * hkv, d)  # the synthetic weights are not trained: to unit size
    pos = ints([n - 1 for n in kv], cuda_device)
    plan = lib.RopePlan(d, d, 10000.0, [64])
    before = qkv.clone()
    lib.bgq_rope(plan, qkv[:, :hq + hkv], pos, y=qkv[:, :hq + hkv])
    cache, seqs = c.cache(), c.seqs()
    lib.bgq_kv4_append(cache, seqs, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])
    out, lse = lib.bgq_kv4_attention(cache, seqs, qkv[:, :hq], want_lse=True)
    y = lib.q4_gemv(mats[1][2], out.reshape(B, hq * d))
    res = h.to(cuda_device).clone()
    lib.bgq_residual_add(res, y.float())
    # every step against the oracle on that step's own inputs
    rope_close(f64(qkv[:, :hq + hkv]), f64(before[:, :hq + hkv]),
               A.rope(f64(before[:, :hq + hkv]), pos.cpu().numpy()[None], d, 10000.0, [64]), 64, False)
    for i, x in ((0, qkv[:, hq:hq + hkv]), (2, qkv[:, hq + hkv:])):
        code, scale, bias, _ = A.kv4_quantise(f64(x))
        for b in range(B):
            p, at = A.slot(kv[b] - 1, b, c.pages, page, c.n_pages)
            c.np[i][p, :, at] = A.kv4_pack(code[b])
            c.np[i + 1][p, :, at] = np.stack([O.f64_to_bf16_bits(scale[b]), O.f64_to_bf16_bits(bias[b])], -1)
    assert np.array_equal(cache.v_q.cpu().numpy().view(np.uint32), c.np[2]) and np.array_equal(bits16(cache.k_sb), c.np[1])
    attn_close(c, qkv[:, :hq], out, lse)
    for b in range(B):
        want = O.gemv(mats[1][0].numpy(), bits16(mats[1][1]), 4, f64(out[b].reshape(-1)))
        assert rel_l2(f64(y[b]), want) <= 2.0 ** -8
    assert torch.equal(res, h.to(cuda_device) + y.float())


# ------------------------------------------------------------------ long lists, shared workspaces, hints
LONG = [dict(kv=[40000], new=[1], hq=4, hkv=1, d=128), dict(kv=[30000], new=[1], hq=16, hkv=1, d=256), dict(kv=[17, 25000], new=[2, 3], hq=10, hkv=1, d=64),
        dict(kv=[20000, 9], new=[3, 1], hq=8, hkv=1, d=128), dict(kv=[24000], new=[5], hq=8, hkv=1, d=256), dict(kv=[30000], new=[9], hq=8, hkv=1, d=64),
        dict(kv=[26000, 70], new=[20, 33], hq=4, hkv=1, d=128)]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 9001)])
@pytest.mark.parametrize("kw", LONG)
def test_units_cut_into_many_parts(cuda_device, kw, causal, window):
    """One or two units that all CTAs share: their parts are joined in two levels (few rows) or by groups of threads."""
    kw = dict(kw)
    hq = kw.pop("hq")
    c = Case(cuda_device, seed=11, page=64, **kw)
    q = bf16(c.rng, c.rows, hq, c.d, dev=cuda_device, scale=1.5)
    cache, seqs = c.cache(), c.seqs()
    out, lse = lib.bgq_kv4_attention(cache, seqs, q, causal=causal, window=window, want_lse=True)
    attn_close(c, q, out, lse, causal=causal, window=window)
    again, _ = lib.bgq_kv4_attention(cache, seqs, q, causal=causal, window=window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (256, 1), (64, 40), (128, 40), (256, 40)])
def test_lse_keeps_single_precision(cuda_device, d, new):
    """Products of codes, scales and queries are exact, and a score is the sum of at most d/16 + 2d/64 + 4 <= 28 partial
    sums in fp32, each off by 2^-23 of itself (truncation): independent errors of terms no larger than the sum add up to
    sqrt(28) 2^-23 |score|, with scores of a few units against an lse of 5 or more below 2^-20 of it. A key rounded to fp16
    would put 2^-12 / sqrt(80) of the score there."""
    c = Case(cuda_device, [80, 75, 66, 71], [new] * 4, 2, d, 16, seed=12)
    q = bf16(c.rng, c.rows, 8, d, dev=cuda_device, scale=1.5)
    _, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    want = c.oracle(q)[1]
    assert rel_l2(f64(lse), want) <= 2.0 ** -20


SHORT = [dict(kv=[200], new=[200], hq=8, hkv=2, d=128, page=64), dict(kv=[311, 150, 129], new=[150, 1, 129], hq=4, hkv=1, d=128, page=16),
         dict(kv=[160, 1000], new=[96, 3], hq=10, hkv=2, d=64, page=32), dict(kv=[140, 260, 0], new=[100, 33, 2], hq=6, hkv=1, d=256, page=64),
         dict(kv=[270], new=[270], hq=3, hkv=1, d=128, page=16, pages=False), dict(kv=[1024, 5], new=[9, 5], hq=64, hkv=8, d=64, page=16),
         dict(kv=[1040, 5], new=[9, 5], hq=64, hkv=8, d=64, page=16), dict(kv=[512], new=[20], hq=8, hkv=8, d=256, page=32)]


@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("kw", SHORT)
def test_many_rows_of_short_page_lists(cuda_device, kw, causal, window):
    """Page lists just long enough: where they hold little, many rows take another kernel than with long ones."""
    kw = dict(kw)
    hq = kw.pop("hq")
    c = Case(cuda_device, seed=18, room=0, gap=1, behind=1, **kw)
    q = bf16(c.rng, c.rows, hq, c.d, dev=cuda_device, scale=1.5)
    out, lse = torch.full_like(q, 7.0), torch.full((c.rows, hq), 7.0, device=cuda_device)
    lib.bgq_kv4_attention(c.cache(), c.seqs(), q, causal=causal, window=window, out=out, lse=lse)
    live = attn_close(c, q, out, lse, causal=causal, window=window)
    dead = torch.from_numpy(~live).to(cuda_device)
    assert (out[dead] == 7.0).all() and (lse[dead] == 7.0).all()


def test_one_workspace_for_all_shapes(cuda_device):
    """Prompts, steps and drafted tokens of different sizes in turn through one workspace give the bits of fresh ones."""
    calls = []
    for i, (kv, new, hq, hkv, d) in enumerate([([300], [300], 8, 2, 128), ([5000], [1], 8, 1, 128), ([900, 70], [1, 1], 8, 2, 64), ([2000], [5], 16, 1, 256),
                                               ([9000], [1], 16, 1, 256), ([130, 64], [100, 64], 4, 2, 64), ([8000, 3], [2, 3], 16, 1, 128)]):
        c = Case(cuda_device, kv, new, hkv, d, 16, seed=20 + i)
        calls.append((c.cache(), c.seqs(), bf16(c.rng, c.rows, hq, d, dev=cuda_device)))
    want = [lib.bgq_kv4_attention(*c, want_lse=True) for c in calls]
    ws = lib.workspace(max(lib.kv4_attention_workspace_bytes(c, s, q.shape[1]) for c, s, q in calls), cuda_device)
    for _ in range(2):
        for c, w in zip(calls, want):
            out, lse = lib.bgq_kv4_attention(*c, want_lse=True, ws=ws)
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    assert lib.read_device_status(ws) == lib.OK


@pytest.mark.parametrize("hint", [1, 4, 1000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_max_q_is_a_hint(cuda_device, d, hint):
    """A sequence with more rows than max_q says is computed all the same, with fewer too."""
    c = Case(cuda_device, [90, 200, 31], [33, 2, 31], 2, d, 48, seed=13)
    q = bf16(c.rng, c.rows, 8, d, dev=cuda_device)
    s = c.seqs()
    out, lse = lib.bgq_kv4_attention(c.cache(), lib.KV4Seqs(s.kv_len, rows=c.rows, pages=s.pages, q_start=s.q_start, max_q=hint), q, want_lse=True)
    attn_close(c, q, out, lse)


@pytest.mark.parametrize("max_q", [1, 64])
def test_no_sequence_has_a_row(cuda_device, max_q):
    """Rows, but none of any sequence: nothing is written."""
    c = Case(cuda_device, [50, 0, 20], [0, 0, 0], 2, 128, 16, behind=9)
    q = bf16(c.rng, 9, 8, 128, dev=cuda_device)
    out = torch.full_like(q, 7.0)
    lse = torch.full((9, 8), 7.0, device=cuda_device)
    s = c.seqs()
    lib.bgq_kv4_attention(c.cache(), lib.KV4Seqs(s.kv_len, rows=9, pages=s.pages, q_start=s.q_start, max_q=max_q), q, out=out, lse=lse)
    assert (out == 7.0).all() and (lse == 7.0).all()


def test_largest_batch(cuda_device):
    """4096 sequences of up to 40 tokens, single rows and (some without any) drafted ones."""
    B = 4096
    kv = [(7 * b) % 41 for b in range(B)]
    for new in ([1] * B, [(b % 7) if kv[b] >= b % 7 else 0 for b in range(B)]):
        c = Case(cuda_device, kv, new, 1, 64, 16, seed=14)
        q = bf16(c.rng, c.rows, 8, 64, dev=cuda_device)
        out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
        attn_close(c, q, out, lse)


@pytest.mark.parametrize("new", [1, 5, 40])
def test_few_of_many_sequences_have_rows(cuda_device, new):
    """Seven of 3000 sequences, runs of up to a thousand without rows between them."""
    at = [3, 4, 40, 900, 1901, 1933, 2999]
    c = Case(cuda_device, [1100 + 37 * (b % 5) if b in at else b % 3 for b in range(3000)], [new if b in at else 0 for b in range(3000)], 2, 64, 16, seed=19)
    q = bf16(c.rng, c.rows, 16, 64, dev=cuda_device)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    attn_close(c, q, out, lse)


def test_two_streams_at_once(cuda_device):
    """Calls that run side by side, with workspaces of their own, give the bits of calls in turn."""
    c = Case(cuda_device, [3000, 800], [1, 1], 2, 128, 16, seed=15)
    p = Case(cuda_device, [700], [700], 2, 128, 16, seed=16)
    jobs = [(x.cache(), x.seqs(), bf16(x.rng, x.rows, 8, 128, dev=cuda_device)) for x in (c, p)]
    want = [lib.bgq_kv4_attention(*j)[0] for j in jobs]
    ws = [lib.workspace(lib.kv4_attention_workspace_bytes(j[0], j[1], 8), cuda_device) for j in jobs]
    outs = [[torch.empty_like(j[2]) for _ in range(8)] for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(8):
        for j, w, o, s in zip(jobs, ws, outs, streams):
            with torch.cuda.stream(s):
                lib.bgq_kv4_attention(*j, out=o[i], ws=w)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)


def test_page_listed_twice_and_short_lists(cuda_device):
    """Two sequences may read the same pages (a shared prefix); tokens beyond a page list are absent."""
    c = Case(cuda_device, [64, 64, 70], [1, 1, 20], 2, 128, 16, seed=17, room=0)
    c.pages[1] = c.pages[0]
    c.kv[2] = 100  # its list has room for 80: rows stand at 80 .. 99
    q = bf16(c.rng, c.rows, 8, 128, dev=cuda_device)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    attn_close(c, q, out, lse)


# ------------------------------------------------------------------ rows far apart
FAR = (1 << 31) + 4096  # values from a row to the next: past 32 bits in values, and in bytes


def far_rows(x):
    """The two rows of x, FAR values apart."""
    big = torch.empty(FAR + x[0].numel(), dtype=BF, device=x.device)
    far = big.as_strided(x.shape, (FAR, x.shape[2], 1))
    far.copy_(x)
    return far


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_rows_far_apart(cuda_device, pairs):
    x = bf16(torch.Generator().manual_seed(30), 2, 5, 64, dev=cuda_device)
    plan, pos = lib.RopePlan(64, 48, 1e4, [24], pairs=pairs), ints([2 ** 31 - 1, -7], cuda_device)
    want = lib.bgq_rope(plan, x, pos)
    far = far_rows(x)
    lib.bgq_rope(plan, far, pos, y=far)
    assert torch.equal(far, want)


@pytest.mark.parametrize("d,max_q,room", [(64, 1, 2048), (128, 1, 2048), (256, 1, 2048), (128, 64, 2048), (256, 64, 2048)])
def test_attention_rows_far_apart(cuda_device, d, max_q, room):
    c = Case(cuda_device, [90, 41], [1, 1], 2, d, 16, seed=31, room=room)
    q, k = bf16(c.rng, 2, 8, d, dev=cuda_device), bf16(c.rng, 2, 2, d, dev=cuda_device)
    s = c.seqs()
    seqs = lib.KV4Seqs(s.kv_len, rows=2, pages=s.pages, q_start=s.q_start, max_q=max_q)
    near, away = c.cache(), c.cache()
    lib.bgq_kv4_append(near, seqs, k, k)
    fk = far_rows(k)
    lib.bgq_kv4_append(away, seqs, fk, fk)
    for name in ("k_q", "k_sb", "v_q", "v_sb"):
        assert torch.equal(getattr(near, name), getattr(away, name))
    back = [far_rows(torch.zeros_like(k)) for _ in range(2)]
    lib.bgq_kv4_read(away, seqs, *back)
    for x, y in zip(back, lib.bgq_kv4_read(near, seqs)):
        assert torch.equal(x, y)
    want, _ = lib.bgq_kv4_attention(near, seqs, q)
    out = far_rows(torch.zeros_like(q))
    lib.bgq_kv4_attention(away, seqs, far_rows(q), out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_around_a_large_offset(cuda_device, d, new):
    """Keys of 60 and a little: scores of thousands whose differences are small. They are off by 2^-22 of the partial sums
    (scale * sum|q k|), probabilities by as much, and by the kernels' own 2^-10."""
    c = Case(cuda_device, [150, 77], [new, new], 1, d, 16, seed=32)
    code, scale, bias, _ = A.kv4_quantise(60 + 0.5 * np.random.default_rng(1).standard_normal((c.n_pages, 1, 16, d)))
    c.np[0], c.np[1] = A.kv4_pack(code).astype(np.uint32), np.stack([O.f64_to_bf16_bits(scale), O.f64_to_bf16_bits(bias)], -1)
    q = bf16(c.rng, c.rows, 8, d, dev=cuda_device)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    o, l, a, s = c.oracle(q)
    e = 2.0 ** -22 * s * (d / 16 + 8)  # every one of the d/16 + 8 partial sums may be off by that
    assert (np.abs(f64(lse) - l) <= e + 2.0 ** -18 * np.abs(l)).all()
    assert (np.abs(f64(out) - o) <= 2.0 ** -8 * np.abs(o) + (2 * e + 2.0 ** -9)[..., None] * a).all()
