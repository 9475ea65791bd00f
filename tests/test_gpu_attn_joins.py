"""Adjacent units of the few-row attention kernel that are both cut into many parts, joined in two levels, against the fp64
oracle: next to each other in one list, repeated on one workspace, and beside another stream's work."""

import pytest
import torch

from bit_group_quantized_gb300 import lib
from tests.test_gpu_attn import Case, attn_close, bf16

pytestmark = pytest.mark.gpu

# the last eight of one unit is a single part, in the CTA where the next unit begins
ADJACENT = [dict(kv=[14197], hq=64, hkv=4, d=256), dict(kv=[20000, 23000], hq=32, hkv=2, d=256), dict(kv=[30000, 30100], hq=16, hkv=1, d=128),
            dict(kv=[9000, 21000, 8000], hq=16, hkv=1, d=256)]


@pytest.mark.parametrize("kw", ADJACENT)
def test_adjacent_units_joined_in_two_levels(cuda_device, kw):
    kw = dict(kw)
    hq = kw.pop("hq")
    c = Case(cuda_device, new=[1] * len(kw["kv"]), page=64, seed=40, **kw)
    q = bf16(c.rng, c.rows, hq, c.d, dev=cuda_device, scale=1.5)
    cache, seqs = c.cache(), c.seqs()
    ws = lib.workspace(lib.kv4_attention_workspace_bytes(cache, seqs, hq), cuda_device)
    out, lse = lib.bgq_kv4_attention(cache, seqs, q, want_lse=True, ws=ws)
    attn_close(c, q, out, lse)
    other = torch.randn(4096, 4096, device=cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = []
    for i in range(24):  # CTAs start at different times where another stream's kernels hold their SMs
        with torch.cuda.stream(side):
            other = torch.tanh(other @ other * 2.0 ** -12)
        again.append(lib.bgq_kv4_attention(cache, seqs, q, want_lse=True, ws=ws))
    torch.cuda.synchronize()
    for o, l in again:
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert not ws[256:4096].any()  # the arrival counters
