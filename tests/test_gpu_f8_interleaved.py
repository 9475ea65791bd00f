"""What a step keeps of each row, side by side in one buffer: the e4m3 calls read and write rows that lie between each other's."""

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib
from tests.test_gpu_f8 import byts, random_matrix

pytestmark = pytest.mark.gpu

U8 = torch.uint8


@pytest.mark.parametrize("m", [1, 5, 70, 300, 20000])
def test_all_of_a_row_side_by_side(cuda_device, m):
    dev, rng, k, n = cuda_device, np.random.default_rng(m), 272, 144
    sizes = dict(x=2 * k, q=k, s=16, h=n, hs=16, y=2 * n)  # bytes of a row
    at, pitch = {}, 0
    for name, size in sizes.items():
        at[name], pitch = pitch, pitch + -(-size // 16) * 16
    pitch = -(-pitch // 256) * 256
    wide = torch.full((m, pitch), 0x55, dtype=U8, device=dev)

    def part(name, dtype, cols):
        return wide[:, at[name]:at[name] + cols * dtype.itemsize].view(dtype)

    x = part("x", torch.bfloat16, k)
    x.copy_(torch.from_numpy(rng.standard_normal((m, k))).bfloat16())
    X = lib.F8Matrix(part("q", lib._F8, k), part("s", lib._E8, 3))
    H = lib.F8Matrix(part("h", lib._F8, n), part("hs", lib._E8, 2))
    y = part("y", torch.bfloat16, n)
    W, _ = random_matrix(dev, rng, n, k, 128, lo=116, hi=119)
    lib.bgq_f8_quantise(x, out=X)
    lib.bgq_f8_swiglu(W, W, X, h=H, out=y)
    near = lib.bgq_f8_quantise(x.contiguous())
    h, out = lib.bgq_f8_swiglu(W, W, near, want_out=True)
    assert np.array_equal(byts(X.q), byts(near.q)) and np.array_equal(byts(X.scale), byts(near.scale))
    assert np.array_equal(byts(H.q), byts(h.q)) and np.array_equal(byts(H.scale), byts(h.scale)) and torch.equal(y, out)
    lib.bgq_f8_gemm(W, X, out=y)
    assert torch.equal(y, lib.bgq_f8_gemm(W, near)[0])
    used = torch.zeros(pitch, dtype=torch.bool)
    for name, size in dict(x=2 * k, q=k, s=3, h=n, hs=2, y=2 * n).items():
        used[at[name]:at[name] + size] = True
    assert (wide[:, ~used] == 0x55).all()
    # and half a row's width further along, over the codes that it reads
    if m > 1:
        with pytest.raises(lib.BGQError):
            lib.bgq_f8_gemm(W, X, out=wide[:, at["q"] - 2 * n + 16:at["q"] + 16].view(torch.bfloat16))
