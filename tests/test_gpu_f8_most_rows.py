"""Products of as many rows as the entry points take."""

import pytest
import torch

from bit_group_quantized_gb300 import lib
from oracle import f8_oracle as F
from tests.f8_rule import kernel
from tests.helpers import f64
from tests.test_gpu_f8 import check_codes, sum_tolerance, swiglu_tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [(1 << 24) - 1, 16776961])
def test_the_most_rows(cuda_device, m):
    """More tiles of 256 rows (gated: 128) than a grid's y has room for."""
    dev, k, n = cuda_device, 16, 16
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert kernel(m, n, k, False, sms) == kernel(m, n, k, True, sms) == "many"
    gen = torch.Generator(device=dev).manual_seed(m)
    q = torch.randint(0, 127, (m, k), dtype=torch.uint8, device=dev, generator=gen)
    s = torch.full((m, 4), 127, dtype=torch.uint8, device=dev)
    X = lib.F8Matrix(q.view(lib._F8), s.view(lib._E8)[:, :1])
    wq = torch.randint(0, 64, (n, k), dtype=torch.uint8, device=dev, generator=gen)  # below 1.875
    W = lib.F8Matrix(wq.view(lib._F8), torch.full((1, 4), 125, dtype=torch.uint8, device=dev).view(lib._E8)[:, :1], 128)
    w = F.values(wq.cpu().numpy(), [[125]], 128)
    y = lib.bgq_f8_gemm(W, X, want_out=False, want_f32=True)[1]
    h, _ = lib.bgq_f8_swiglu(W, W, X)
    last = m // 256 * 256
    for rows in (slice(0, 300), slice(65535 * 128 - 100, 65535 * 128 + 100), slice(last - 200, m)):
        x = F.values(q[rows].cpu().numpy(), [[127]] * len(range(*rows.indices(m))))
        ref, size = F.product(x, w)
        assert (abs(f64(y[rows]) - ref) <= sum_tolerance(size, k)).all()
        check_codes(lib.F8Matrix(h.q[rows], h.scale[rows]), F.swiglu(ref, ref), swiglu_tolerance(ref, ref, size, size, k))
