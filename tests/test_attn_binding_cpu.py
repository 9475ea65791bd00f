"""What the binding of the attention operators refuses before it calls the library, without a GPU."""

import types

import pytest
import torch

from bit_group_quantized_gb300 import lib


def test_streams_of_another_device_are_refused():
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(lib.BGQError) as e:
        lib._there(0, other)
    assert e.value.status == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("args", [(2 ** 32 + 128, 128, 1e4, [64]), (128, 2 ** 32 + 128, 1e4, [64]), (128, 128, 1e4, [2 ** 32 + 64]),
                                  (128, 128, 1e4, [64, -2 ** 32])])
def test_rope_plan_numbers_beyond_32_bits(args):
    with pytest.raises(lib.BGQError) as e:
        lib.RopePlan(*args)
    assert e.value.status == lib.ERR_INVALID_ARG


def test_numbers_beyond_32_bits():
    for v in (2 ** 31, 2 ** 32, -2 ** 31 - 1):
        with pytest.raises(lib.BGQError):
            lib._int32(v, "it")
    assert lib._int32(2 ** 31 - 1, "it") == 2 ** 31 - 1
