"""csrc/f8_rule.h compiled for the host: which kernel a product of e4m3 matrices takes, and how it is cut."""

import ctypes as C
import functools
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc")
SMS = 152  # of one GB300

SOURCE = r"""
#include "f8_rule.h"
using namespace bgq;
extern "C" int f8_choice(int m, int n, int k, int gated, int sms, int* plan, double* us) {
  const F8Size s = {m, n, k, gated != 0};
  const F8MidPlan mid = f8_mid_plan(s, sms);
  plan[0] = mid.down, plan[1] = mid.rows, plan[2] = mid.split;
  plan[3] = gated ? 256 : f8_many_wide(s, sms / 2);
  us[0] = f8_few_us(s), us[1] = mid.us, us[2] = f8_many_us(s, sms);
  return (int)f8_kernel(s, sms, mid);
}
"""


@functools.lru_cache(None)
def _lib():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no host compiler")
    at = tempfile.mkdtemp()
    src, out = os.path.join(at, "rule.cpp"), os.path.join(at, "rule.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-shared", "-fPIC", "-I", CSRC, src, "-o", out], check=True)
    lib = C.CDLL(out)
    shutil.rmtree(at)
    return lib


class Choice:
    """kernel: 'few', 'mid' or 'many'; a batch's plan (tiles of x's rows, rows of each, shares of the columns); rows of W a
    tile of the kernel for many rows; the three estimates."""

    def __init__(self, m, n, k, gated=False, sms=SMS):
        plan, us = (C.c_int * 4)(), (C.c_double * 3)()
        self.kernel = ("few", "mid", "many")[_lib().f8_choice(m, n, k, gated, sms, plan, us)]
        self.down, self.rows, self.split, self.wide = plan
        self.few_us, self.mid_us, self.many_us = us


def kernel(m, n, k, gated=False, sms=SMS):
    return Choice(m, n, k, gated, sms).kernel
