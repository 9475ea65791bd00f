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
