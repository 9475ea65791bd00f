"""Attention with windows that hide nothing, up to 2^31 - 1: the bits of a call without one."""

import pytest
import torch

from bit_group_quantized_gb300 import lib
from tests.test_gpu_attn import Case, attn_close, bf16

pytestmark = pytest.mark.gpu

# more rows than tokens (rows at negative positions), a single token a sequence, drafted rows, a last block cut short
SEQS = [dict(kv=[3, 40], new=[9, 5], hq=4, hkv=2, d=128), dict(kv=[70, 1, 300], new=[1, 1, 1], hq=8, hkv=2, d=64), dict(kv=[45, 6], new=[8, 30], hq=8, hkv=1, d=256),
        dict(kv=[61, 333, 20], new=[61, 90, 45], hq=8, hkv=2, d=128), dict(kv=[150, 10], new=[70, 40], hq=4, hkv=1, d=256)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kw", SEQS)
def test_large_windows_hide_nothing(cuda_device, kw, causal):
    kw = dict(kw)
    hq = kw.pop("hq")
    c = Case(cuda_device, page=16, seed=41, **kw)
    q = bf16(c.rng, c.rows, hq, c.d, dev=cuda_device, scale=1.5)
    cache, seqs = c.cache(), c.seqs()
    out, lse = lib.bgq_kv4_attention(cache, seqs, q, causal=causal, want_lse=True)
    attn_close(c, q, out, lse, causal=causal)
    for window in (2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30):
        o, l = lib.bgq_kv4_attention(cache, seqs, q, causal=causal, window=window, want_lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse), window


@pytest.mark.parametrize("new", [1, 40])
def test_length_far_beyond_the_page_list(cuda_device, new):
    """A length near 2^31 over a list that ends long before: tokens that it does not hold are absent, and with a window that
    begins behind the list no row sees any."""
    c = Case(cuda_device, [96], [new], 2, 128, 16, seed=42)
    q = bf16(c.rng, c.rows, 8, 128, dev=cuda_device)
    cache, seqs = c.cache(), c.seqs()
    for length in (2 ** 31 - 1, 2 ** 31 - 65536, 2 ** 31 - 70000):
        seqs.kv_len.fill_(length)
        o, l = lib.bgq_kv4_attention(cache, seqs, q, window=1, want_lse=True)
        assert not o.any() and torch.isneginf(l).all()
        o, l = lib.bgq_kv4_attention(cache, seqs, q, causal=False, want_lse=True)
        attn_close(c, q, o, l, causal=False)


@pytest.mark.parametrize("max_q", [1, 64])
@pytest.mark.parametrize("first,end", [(0, 2 ** 29), (0, 2 ** 31 - 1), (1, 2 ** 30 + 1), (-(2 ** 31), 2 ** 31 - 1)])
def test_sequences_of_more_rows_than_the_call_has(cuda_device, max_q, first, end):
    """Row starts far beyond the rows: the rows there are belong to the sequence, at the negative positions that its length gives them,
    where they see nothing; with a mask that hides none they see all."""
    c = Case(cuda_device, [96], [3], 2, 128, 16, seed=43, behind=2)
    q = bf16(c.rng, c.rows, 8, 128, dev=cuda_device)
    s = c.seqs()
    seqs = lib.KV4Seqs(s.kv_len, rows=c.rows, pages=s.pages, q_start=torch.tensor([first, end], dtype=torch.int32, device=cuda_device), max_q=max_q)
    out, lse = torch.full_like(q, 7.0), torch.full((c.rows, 8), 7.0, device=cuda_device)
    lib.bgq_kv4_attention(c.cache(), seqs, q, out=out, lse=lse)
    own = slice(max(first, 0), c.rows) if first > -2 ** 31 else slice(0, 0)  # 2^32 - 1 rows are none that a position has
    assert not out[own].any() and torch.isneginf(lse[own]).all()
    assert (out[:own.start] == 7.0).all()
    if first < 0:
        return
    lib.bgq_kv4_attention(c.cache(), seqs, q, causal=False, out=out, lse=lse)
    c.q_start = [first, c.rows]
    attn_close(c, q, out, lse, causal=False)
