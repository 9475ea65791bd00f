"""The gated half of a feed-forward block where a gate lies so far below zero that its exponential leaves fp32: the product with a
large other half is still an ordinary number. For each of the three kernels, which the test names."""

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib
from oracle import f8_oracle as F
from tests.f8_rule import kernel
from tests.helpers import f64
from tests.test_gpu_f8 import check_codes, matrix

pytestmark = pytest.mark.gpu

# gates: -1 to -448 in every code, and their opposites
GATES = np.concatenate([np.arange(0xb8, 0xff), np.arange(0x38, 0x7f)]).astype(np.uint8)
CASES = [("few", 2), ("few", 7), ("mid", 40), ("mid", 500), ("many", 26000)]


@pytest.mark.parametrize("up", [100, 20, 0, -60])
@pytest.mark.parametrize("name,m", CASES)
def test_far_gates(cuda_device, name, m, up):
    k, n = 16, 16 * 18  # of which the last 2 hold zeros
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert kernel(m, n, k, True, sms) == name
    x = np.zeros((m, k), dtype=np.uint8)
    x[:, 0] = 0x38  # 1
    g, u = np.zeros((n, k), dtype=np.uint8), np.zeros((n, k), dtype=np.uint8)
    g[:142, 0], g[142:284, 0] = GATES, GATES[::-1]
    u[:142, 0], u[142:284, 0] = 0x39, 0xbc  # 1.125 and -1.5
    X = matrix(cuda_device, x, np.full((m, 1), 127, dtype=np.uint8), 1)
    G = matrix(cuda_device, g, np.full((3, 1), 127, dtype=np.uint8), 128)
    U = matrix(cuda_device, u, np.full((3, 1), 127 + up, dtype=np.uint8), 128)
    gate, other = F.values(g, np.full((3, 1), 127, dtype=np.uint8), 128)[:, 0], F.values(u, np.full((3, 1), 127.0 + up), 128)[:, 0]
    ref = F.swiglu(gate, other)
    # g and u are exact. Down to -64 the exponential is off by 2 + 1.2 |g| units of 2^-23, the reciprocal and the products by one
    # each. Below, that of -64 is multiplied by the square of 2^a, a = (g + 64) / 2 * log2(e): a is rounded once and its constant once, each by
    # 2^-24 |a| at most: log(2) times both is 0.5 |g + 64| units of 2^-23 in each of two factors. Each power is off by two units besides,
    # and four products by half of one.
    far = np.maximum(-64 - gate, 0)
    off = np.abs(ref) * (8 + 1.2 * np.minimum(np.abs(gate), 64) + np.where(far > 0, 6 + far, 0)) * 2.0 ** -23 + 2.0 ** -149
    h, y = lib.bgq_f8_swiglu(G, U, X, want_out=True)
    got = f64(y)
    assert (got == got[0]).all()
    bad = ~(np.abs(got[0] - ref) <= off + (np.abs(ref) + off) * 2.0 ** -8 + 2.0 ** -134)
    assert not bad.any(), [(gate[i], other[i], got[0, i], ref[i]) for i in np.flatnonzero(bad)[:5]]
    rows = slice(0, m, max(1, m // 40))
    check_codes(lib.F8Matrix(h.q[rows].contiguous(), _scales(h, rows)), np.tile(ref, (len(range(*rows.indices(m))), 1)), np.tile(off, (len(range(*rows.indices(m))), 1)))


def _scales(h, rows):
    part = h.scale[rows]
    out = lib.F8Matrix.empty_scale(part.shape[0], h.cols, part.device)
    out.view(torch.uint8).copy_(part.view(torch.uint8))
    return out
