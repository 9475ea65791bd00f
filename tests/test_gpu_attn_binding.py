"""What the binding of the attention operators refuses, and takes, on a GPU."""

import pytest
import torch

from bit_group_quantized_gb300 import lib
from tests.test_gpu_attn import Case, bf16

pytestmark = pytest.mark.gpu


def test_numbers_beyond_32_bits_are_refused(cuda_device):
    """A window of 2^32 + 5 is not one of 5."""
    c = Case(cuda_device, [50], [1], 2, 64, 16, seed=60)
    q = bf16(c.rng, 1, 4, 64, dev=cuda_device)
    cache, seqs = c.cache(), c.seqs()
    for window in (2 ** 31, 2 ** 32 + 5):
        with pytest.raises(lib.BGQError) as e:
            lib.bgq_kv4_attention(cache, seqs, q, window=window)
        assert e.value.status == lib.ERR_INVALID_ARG
    for kw in (dict(rows=2 ** 32 + 1), dict(rows=1, max_q=2 ** 32 + 1)):
        with pytest.raises(lib.BGQError):
            lib.KV4Seqs(seqs.kv_len, pages=seqs.pages, q_start=seqs.q_start, **kw)
    with pytest.raises(lib.BGQError):
        lib.kv4_attention_workspace_bytes(cache, seqs, 2 ** 32 + 4)


def test_a_workspace_that_only_seems_large_is_refused(cuda_device):
    """An expanded tensor has the bytes of its shape to its name, not to its memory; a strided one has holes that belong to others."""
    c = Case(cuda_device, [50], [1], 2, 64, 16, seed=61)
    q = bf16(c.rng, 1, 4, 64, dev=cuda_device)
    cache, seqs = c.cache(), c.seqs()
    need = lib.kv4_attention_workspace_bytes(cache, seqs, 4)
    for ws in (torch.zeros(256, dtype=torch.uint8, device=cuda_device)[:1].expand(need), torch.zeros(2 * need, dtype=torch.uint8, device=cuda_device)[::2]):
        with pytest.raises(lib.BGQError) as e:
            lib.bgq_kv4_attention(cache, seqs, q, ws=ws)
        assert e.value.status == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("tokens", [1, 40])
def test_rope_positions_shared_by_all_axes(cuda_device, tokens):
    """Positions of plain text, expanded over the axes: the bits of a copy for each."""
    rng = torch.Generator().manual_seed(62)
    x = bf16(rng, tokens, 3, 64, dev=cuda_device)
    plan = lib.RopePlan(64, 64, 10000.0, [12, 10, 10])
    pos = torch.randint(0, 5000, (tokens,), generator=rng, dtype=torch.int32).to(cuda_device)
    want = lib.bgq_rope(plan, x, pos.repeat(3, 1))
    assert torch.equal(lib.bgq_rope(plan, x, pos.expand(3, tokens)), want)


@pytest.mark.parametrize("kv,new,hq,hkv,d", [([700], [700], 8, 2, 128), ([3000, 90], [1, 1], 8, 2, 64), ([20000], [1], 16, 1, 256), ([900, 40], [33, 5], 8, 1, 256)])
def test_only_the_head_of_a_workspace_is_zero_filled(cuda_device, guard_canaries, kv, new, hq, hkv, d):
    """Calls do with any bytes behind the first 4096, and a call without a workspace fills no large one."""
    c = Case(cuda_device, kv, new, hkv, d, 16, seed=63)
    q = bf16(c.rng, c.rows, hq, d, dev=cuda_device)
    cache, seqs = c.cache(), c.seqs()
    asked = []

    def allocator(shape, dtype, device, zero):
        asked.append((torch.empty(0, dtype=dtype).element_size() * torch.Size(shape).numel(), zero))
        return guard_canaries(shape, dtype, device, zero)

    lib.set_allocator(allocator)
    want, lse = lib.bgq_kv4_attention(cache, seqs, q, want_lse=True)
    assert max(n for n, _ in asked) > 4096 and all(n <= 8 << 20 for n, zero in asked if zero)
    ws = lib.kv4_attention_workspace(cache, seqs, hq)
    for fill in (0xff, 0x7f, 0x01):
        ws[4096:] = fill
        for _ in range(2):
            out, l = lib.bgq_kv4_attention(cache, seqs, q, want_lse=True, ws=ws)
            assert torch.equal(out, want) and torch.equal(l, lse)
    assert lib.read_device_status(ws) == lib.OK


@pytest.mark.parametrize("new", [1, 60])
def test_an_output_in_the_queries_place_is_refused(cuda_device, new):
    """A row's heads are read by other blocks than the one that writes them."""
    c = Case(cuda_device, [80], [new], 2, 64, 16, seed=64)
    q = bf16(c.rng, new, 4, 64, dev=cuda_device)
    with pytest.raises(lib.BGQError) as e:
        lib.bgq_kv4_attention(c.cache(), c.seqs(), q, out=q)
    assert e.value.status == lib.ERR_INVALID_ARG
