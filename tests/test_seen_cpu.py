"""Which tokens a row of attention sees (csrc/kv4_seen.h), compiled for the host and compared with the definition over
windows, positions and lengths up to the ends of their 32 bits."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc")

HARNESS = r"""
#include <algorithm>
#include <cstdlib>
#include <vector>
#include "kv4_seen.h"
using namespace bgq;
typedef __int128 wide;

int main() {
  const int top = 2147483647;
  std::vector<int> edge = {0, 1, 2, 15, 16, 40, 4096, top / 2, top - 65535, top - 4, top - 3, top - 1, top};
  std::vector<int> pos = edge;
  for (int e : edge) pos.push_back(e == 0 ? -top - 1 : -e);
  srand(3);
  for (int i = 0; i < 40; ++i) edge.push_back(rand());
  for (int i = 0; i < 40; ++i) pos.push_back(rand() - rand());
  for (int p : pos)
    for (int w : edge) {
      // the smallest t >= 0 with t > p - w
      const wide first = w > 0 ? std::max((wide)0, (wide)p - w + 1) : 0;
      if (kv4_first_seen(p, w) != first) return 1;
      for (int n : edge)
        for (int held : {0, 1, 17, n}) {
          if (held > n || p >= n) continue;  // a row stands before its sequence's end
          for (int causal : {0, 1}) {
            const wide end = std::max((wide)0, std::min((wide)held, causal ? (wide)p + 1 : (wide)n));
            if (kv4_end_seen(p, n, held, causal) != end) return 2;
          }
        }
    }
  return 0;
}
"""


def test_tokens_seen_at_the_ends_of_32_bits(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "seen.cpp"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(tmp_path / "seen")], check=True)
    assert subprocess.run([str(tmp_path / "seen")]).returncode == 0


def test_kernels_take_their_bounds_from_there():
    """No kernel forms pos - window by itself."""
    for name in ("kv4_split.cu", "kv4_prompt.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert "kv4_first_seen(" in text and "kv4_end_seen(" in text
        assert "- a.window" not in text
