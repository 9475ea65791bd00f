"""Rules that the attention operators state and keep, without a GPU."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc")


def text(*path):
    return open(os.path.join(ROOT, *path), encoding="utf-8").read()


def test_a_page_is_not_offered_as_weights():
    """GEMVs read codes and scales ahead of their wait for earlier kernels; the cache is what an earlier kernel writes."""
    gemv = text("bit_group_quantized_gb300", "csrc", "gemv.cu")
    assert "pdl_wait();" in gemv
    header = text("include", "bgq.h")
    assert "is a bgq_qmatrix" not in header
    about = header[header.index("A paged cache of keys and values in 4 bits"):header.index("typedef struct bgq_kv4_cache")]
    assert re.search(r"must not be given to a call\s*\*?\s*as its weights", about)
    rules = header[header.index("Conventions for every entry point"):header.index("#ifndef BGQ_H")]
    assert "Weights (every bgq_qmatrix, expert and layer) are constants" in rules


def test_no_read_only_loads_of_what_earlier_kernels_write():
    """The kernels start while the one before still runs, so nothing that they read is constant for as long as they live."""
    for name in ("kv4.cu", "kv4_split.cu", "kv4_prompt.cu", "rope.cu", "attn.h"):
        code = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
        assert "__ldg" not in code and "ldg_stream" not in code and "global.nc" not in code, name
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", code), name


def test_rotary_frequencies_keep_the_stated_bound():
    """A plan's frequencies against 60 digits: off by at most 2^-54 of a turn, which is what the header says of a position."""
    import math
    from decimal import Decimal, getcontext

    from bit_group_quantized_gb300 import build, lib

    build.build()
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    for theta in (1.0, 1.5, 100.0, 10000.0, 5e5, 1e6, 1e12):
        ln = Decimal(theta).ln()
        for rot in (16, 96, 128, 256):
            plan = lib.RopePlan(256, rot, theta, [rot // 2]).c
            for i in range(rot // 2):
                turn = (-(Decimal(2 * i) / Decimal(rot)) * ln).exp() / (2 * pi)
                off = abs(Decimal(int(plan.freq[i])) / Decimal(2) ** 64 - turn)
                assert off <= Decimal(2) ** -54, (theta, rot, i, math.log2(off))
    header = text("include", "bgq.h")
    assert "|pos| * 2^-54 turns" in header and "exact at any" not in header
    assert "far positions lose nothing" not in text("bit_group_quantized_gb300", "csrc", "rope.cu")
