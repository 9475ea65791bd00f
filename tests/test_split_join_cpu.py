"""The few-row attention kernel's arithmetic of cut units (csrc/split_join.h), compiled for the host: over lists of
sequences of any lengths, which parts are joined by whom, and that no two joins count at the same place."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "bit_group_quantized_gb300", "csrc", "split_join.h")

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>
#include "%s"
using namespace bgq;

// A list of units (tiles of each), shared out as the kernel does. Returns how many units were joined in two levels; -1: a fault.
static int check(const std::vector<int>& tiles, int grid, int columns, int d) {
  const int cost = 20;
  long long total = 0;
  for (int t : tiles) total += t + cost;
  long long ctas = total / (8 + cost);
  if (ctas > grid) ctas = grid;
  if (ctas < 1) ctas = 1;
  std::set<int> used;  // every join's counter
  int two = 0;
  long long at = 0;
  for (int t : tiles) {
    const int c0 = split_cta(at + cost, ctas, total), c1 = split_cta(at + cost + t - 1, ctas, total);
    for (int i : {0, t / 2, t - 1}) {  // a place belongs to the CTA whose share holds it
      const long long x = at + cost + i, c = split_cta(x, ctas, total);
      if (x < total * c / ctas || x >= total * (c + 1) / ctas) return -1;
    }
    at += t + cost;
    if (c0 == c1) continue;
    const bool eights = split_two_levels(c1 - c0 + 1, columns, d);
    const SplitJoin all = split_all(c0, c1, eights);
    if (all.counter < 0 || all.counter >= grid || !used.insert(all.counter).second) return -1;
    std::vector<int> joined(c1 - c0 + 1, 0);
    if (!eights) {
      if (all.first != 0 || all.step != 1 || all.n != c1 - c0 + 1) return -1;
      continue;
    }
    ++two;
    int tops = 0;
    for (int c = c0; c <= c1; ++c) {
      const SplitJoin j = split_eight(c0, c1, c, grid);
      if (j.step != 1 || c - c0 < j.first || c - c0 >= j.first + j.n || c0 + j.first + j.n - 1 > c1) return -1;
      if (c - c0 != j.first) continue;  // seen with the eight's first CTA
      for (int i = 0; i < j.n; ++i) ++joined[j.first + i];
      if (j.first != all.first + tops * all.step) return -1;
      ++tops;
      if ((j.counter < 0) != (j.n == 1)) return -1;
      if (j.counter >= 0 && (j.counter < grid || j.counter >= 2 * grid || !used.insert(j.counter).second)) return -1;
    }
    if (tops != all.n) return -1;
    for (int n : joined)
      if (n != 1) return -1;
  }
  return two;
}

int main() {
  // two units of 33 parts, the second beginning where the first one ends; two sequences of 20000 and 23000 tokens
  if (check(std::vector<int>(4, (14197 + 15) / 16), 152, 16, 256) < 2) return 1;
  if (check({1250, 1250, 1438, 1438}, 152, 16, 256) < 2) return 2;
  srand(7);
  int two = 0;
  for (int n = 0; n < 20000; ++n) {
    const int d = 64 << rand() %% 3, columns = 1 + rand() %% 16, grid = (rand() %% 2 ? 152 : rand() %% 2 ? 148 : 132) * (d < 256 ? 1 + rand() %% 2 : 1);
    const int seqs = 1 + rand() %% 6, most = 1 << (4 + rand() %% 14);
    std::vector<int> tiles;
    for (int s = 0; s < seqs; ++s) {
      const int t = 1 + rand() %% most, units = 1 + rand() %% 4;
      tiles.insert(tiles.end(), units, t);
    }
    const int r = check(tiles, grid, columns, d);
    if (r < 0) return 3;
    two += r;
  }
  return two > 1000 ? 0 : 4;
}
"""


def test_joins_of_cut_units_do_not_share_a_counter(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "joins.cpp"
    src.write_text(HARNESS % HEADER)
    subprocess.run([cxx, "-O1", "-std=c++17", str(src), "-o", str(tmp_path / "joins")], check=True)
    assert subprocess.run([str(tmp_path / "joins")]).returncode == 0
