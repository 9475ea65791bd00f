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


def test_rows_of_very_large_scores_pin():
    """A row's scores of 2^30: fp32's products and their maximum, rounded, are that far from the exact ones."""
    s, c = np.float32(3.0000007e9), np.float32(0.1275)
    assert abs(float(s) * float(c) - float(s * c)) > 1  # so exp2 of a fused difference is not 1 at the maximum


@pytest.mark.parametrize("new", [1, 5, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8, 1e16, -1e8])
def test_very_large_scores(cuda_device, d, new, size):
    """Scores of thousands to 1e16 and more, of either sign: the row is its best token's value. A score is off by 2^-13 of scale sum|q k| at
    most: the few-row kernel multiplies 64 + code, whose partial sums in a group reach 21 times sum|q k| (64 |sum q| + 15 sum|q| <= 64 * 28 +
    15 * 51 against 51 * 2.4, in units of the group's scale), and d / 16 + 8 <= 24 of them are each off by 2^-23 of themselves. Rows whose
    best two are nearer than twice that, and 30 for the others' weight, are passed over."""
    c = Case(cuda_device, [300], [new], 1, d, 16, seed=71, room=0 if new == 1 else 2048)
    scale = float(size) * d ** -0.5
    q = torch.randn(c.rows, 4, d, generator=c.rng).to(BF).to(cuda_device)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, scale=scale, want_lse=True)
    from oracle import attn_oracle as A
    k, v = (A.kv4_values(c.np[i], c.np[i + 1]) for i in (0, 2))
    at = [A.slot(t, 0, c.pages, c.page, c.n_pages) for t in range(300)]
    K, V = (np.stack([x[p, 0, o] for p, o in at]) for x in (k, v))
    qd = O.bf16_to_f64(q.cpu().view(torch.int16).numpy().astype(np.uint16))
    got, gl = O.bf16_to_f64(out.cpu().view(torch.int16).numpy().astype(np.uint16)), lse.cpu().double().numpy()
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    checked = 0
    for j in range(new):
        n = 300 - new + j + 1
        for h in range(4):
            s = K[:n] @ qd[j, h] * scale
            off = 2.0 ** -13 * (np.abs(K[:n]) @ np.abs(qd[j, h]) * abs(scale)).max()
            best = int(s.argmax())
            assert abs(gl[j, h] - s[best]) <= off + 2.0 ** -23 * abs(s[best]) + np.log(n)
            if np.sort(s)[-1] - np.sort(s)[-2] > 2 * off + 30:
                # one rounding of the value to bf16 and its own in fp16: code - 8 times the scale, or the value
                assert (np.abs(got[j, h] - V[best]) <= 2.0 ** -8 * np.abs(V[best]) + 2.0 ** -9).all()
                checked += 1
    assert checked > 0
