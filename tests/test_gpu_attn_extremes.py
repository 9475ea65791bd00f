"""Attention with queries at the end of bf16's range: finite values whose scores are ordinary ones, as the keys are small."""

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib
from oracle import bgq_oracle as O
from tests.test_gpu_attn import BF, Case, attn_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 5, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_largest_queries(cuda_device, d, new):
    c = Case(cuda_device, [140], [new], 2, d, 16, seed=70)
    c.np[1] = O.f64_to_bf16_bits(O.bf16_to_f64(c.np[1]) * 2.0 ** -118)
    q = torch.randn(c.rows, 4, d, generator=c.rng)
    q = (torch.sign(q) * q.abs().clamp(0.01, 1.9)).double().mul(2.0 ** 127).to(BF).to(cuda_device)
    assert torch.isfinite(q).all() and float(q.abs().max()) > 3e38
    scale = 2.0 ** -12 * d ** -0.5
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, scale=scale, want_lse=True)
    attn_close(c, q, out, lse, scale=scale)
    # a key of zeros: a score of zero, however large the query
    c.np[1] = np.zeros_like(c.np[1])
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, scale=100.0, want_lse=True)
    attn_close(c, q, out, lse, scale=100.0)
