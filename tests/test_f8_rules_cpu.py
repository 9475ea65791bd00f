"""Rules that the e4m3 operators state and keep, without a GPU."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc")
FILES = ("f8.h", "f8_tc.cuh", "f8_quant.cu", "f8_few.cu", "f8_mid.cu", "f8_many.cu")


def code(name):
    return re.sub(r"//.*", "", open(os.path.join(CSRC, name), encoding="utf-8").read())


def test_no_read_only_loads_of_what_earlier_kernels_write():
    """The kernels start while the one before still runs, weights may be what it writes, and so nothing that they read is
    constant for as long as they live."""
    for name in FILES:
        text = code(name)
        assert "__ldg" not in text and "ldg_stream" not in text and "global.nc" not in text, name
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", text), name


def test_nothing_is_read_before_the_wait():
    """Ahead of pdl_wait() a kernel sets up barriers and tells L2 what it will read, no more."""
    for name in FILES[2:]:
        text = code(name)
        kernels = re.split(r"__global__", text)[1:]
        assert kernels, name
        for k in kernels:
            ahead = k[:k.index("pdl_wait();")]
            assert "reinterpret_cast<const" not in ahead.replace("reinterpret_cast<const uint8_t*>(this)", "") and "f8_load<" not in ahead, name
            assert "ld.global" not in ahead and "cp.async.bulk.tensor" not in ahead and "tmem_alloc" not in ahead, name
            assert k.index("pdl_trigger();") > k.index("pdl_wait();"), name


def test_waits_are_bounded():
    for name in FILES:
        text = code(name)
        assert not re.search(r"while\s*\(\s*!?\s*tc_mbar_try\b", text), name
        for loop in re.findall(r"while \(!tc_mbar_try_suspend[^{]*\{(.*?)\n  \}", text, flags=re.S):
            assert "kF8TimeoutNs" in loop and "it >" in loop, name
