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
