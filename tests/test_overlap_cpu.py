"""csrc/overlap.h, compiled for the host, against the bytes of both arrays one by one."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc")

HARNESS = r"""
#include <cstdlib>
#include <set>
#include "overlap.h"
using namespace bgq;

static bool meet(const Rows& a, const Rows& b) {
  std::set<uintptr_t> bytes;
  for (int64_t i = 0; i < a.rows; ++i)
    for (int64_t k = 0; k < a.width; ++k) bytes.insert((uintptr_t)a.at + i * a.stride + k);
  for (int64_t i = 0; i < b.rows; ++i)
    for (int64_t k = 0; k < b.width; ++k)
      if (bytes.count((uintptr_t)b.at + i * b.stride + k)) return true;
  return false;
}
static int any(int lo, int hi) { return lo + rand() % (hi - lo + 1); }
static Rows some(bool wide) {
  Rows r;
  r.rows = any(0, 7);
  r.width = any(1, 12);
  r.stride = r.width + (wide ? any(0, 24) : 0);
  r.at = (const void*)(uintptr_t)any(1000, 1120);
  return r;
}

int main() {
  srand(7);
  int same = 0, refused = 0, free_ = 0;
  for (int n = 0; n < 200000; ++n) {
    Rows a = some(n & 1), b = some(n & 2);
    if (n % 3 == 0) b.stride = a.stride = a.stride > b.stride ? a.stride : b.stride;
    const bool want = meet(a, b), got = overlap(a, b);
    if (overlap(b, a) != got) return 1;
    if (want && !got) return 2;                                        // never let through
    if (got && !want && a.stride == b.stride) return 3;                // exact at the same distance,
    if (got && !want && (a.rows == 1 || b.rows == 1)) return 4;        // and beside a single row
    if (got && !want && a.stride == a.width && b.stride == b.width) return 5;  // and where both are contiguous
    same += want == got;
    refused += got;
    free_ += !got;
  }
  if (refused < 20000 || free_ < 20000 || same < 190000) return 6;
  // far apart, near the ends of what strides and rows may be, and no address at all
  const Rows big = {(const void*)4096, (1 << 24) - 1, 65536, (int64_t)1 << 36};
  const Rows in = {(const void*)(4096 + ((uint64_t)1 << 50)), 1, 1, 16}, gap = {(const void*)(4096 + ((uint64_t)1 << 50) + 65536), 1, 1, 16};
  if (!overlap(big, in) || overlap(big, gap) || overlap(big, Rows{nullptr, 1, 1, 1})) return 7;
  const Rows a = {(const void*)256, 4, 8, 16}, b = {(const void*)264, 4, 8, 16}, c = {(const void*)260, 4, 8, 16};
  if (overlap({a, b}, {}) || !overlap({a, c}, {}) || overlap({a}, {b}) || !overlap({a}, {b, c}) || overlap({a}, {})) return 8;
  return 0;
}
"""


def test_overlaps_byte_by_byte(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "overlap.cpp"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(tmp_path / "overlap")], check=True)
    assert subprocess.run([str(tmp_path / "overlap")]).returncode == 0
