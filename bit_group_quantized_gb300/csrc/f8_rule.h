// f8_rule.h — which kernel multiplies two e4m3 matrices, and how it cuts them, by sizes alone.
// Plain C++, so that the host can check the arithmetic as the launches run it, and a test can name the kernel that it means.
//
// Three read the same operands and give the same kinds of results:
//   f8_few.cu   few rows, mma.sync, W straight into registers: next to nothing besides W's bytes, which come at 4.4 TB/s;
//   f8_mid.cu   W as the tensor cores' operand of 128 rows, columns split over CTAs: 3 us besides W's bytes at 6.5 TB/s;
//   f8_many.cu  tiles of 256 x 256: 5 us besides, and the most arithmetic a second.
// The one that the estimates call soonest. Measured (CUDA graphs of 24 calls over 130 to 300 MB of
// weights; us, N x K, gated: 2 N x K):
//                     rows:     1     8    16    32    64   128   256   512  1024  2048
//   4096 x 4096       few     4.3   4.7   5.9   8.6  15.9
//                     mid     6.0   6.1   6.2   6.3   7.0   8.0  11.0  14.6  18.0
//                     many                          12.3  12.9  12.9  13.6  16.4  25.3
//   12288 x 4096      few    11.8  12.2  15.0  23.3
//                     mid    11.1  11.1  11.2  11.3  11.8  13.7  19.0
//                     many                          14.8  15.1  15.4  23.8  35.1  64.2
//   4096 x 1024       few     3.2   3.3   3.3   3.5   5.8
//                     mid     3.5   3.5   3.6   3.8   4.4   5.0   4.9   6.2   9.0
//                     many                    5.9   6.0   6.2   6.2   6.7   8.2  11.9
//   1024 x 1024       few     2.1   2.2   2.2   2.5   2.6
//                     mid     3.0   3.0   3.1   3.1   3.5   3.8   4.3
//   256 x 16384       few     7.7   8.5  11.3  19.4
//                     mid     6.0   6.2   6.3   6.7
//   1024 x 4096       few     5.0   5.4   8.9  12.8
//   gated             mid     4.5   4.7   4.8   5.5   6.5   7.1   9.0  11.5  15.6
//                     many                          14.4  14.8  14.8  15.2  15.8  17.4
//   512 x 1024        few     2.9   3.0   3.8   5.8
//   gated             mid     3.5   3.6   3.7   3.8
//   12288 x 4096      few    24.9  25.2  36.6  57.5
//   gated             mid    18.7  18.8  19.2  20.0  22.3  26.2  45.1
//                     many                          28.4  28.7  29.3  38.5  67.3   121
#pragma once

#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <limits>

namespace bgq {

constexpr int kF8Block = 128;  // columns that share one scale (of weights, rows too)

struct F8Size {
  int M, N, K;  // rows of x, rows of W (gated: of gate, and as many of up), columns of both
  bool gated;
};

inline int f8_ceil_div(int a, int b) { return (a + b - 1) / b; }
inline int64_t f8_ceil_div(int64_t a, int b) { return (a + b - 1) / b; }
inline double f8_weights(const F8Size& s) { return (double)s.N * s.K * (s.gated ? 2e-6 : 1e-6); }  // millions of bytes

// ----------------------------------------------------------------- few rows
// Microseconds: a warp's blocks of columns one after the other, or W's bytes.
inline double f8_few_us(const F8Size& s) {
  const int tokens = s.M <= 8 ? 0 : s.M <= 16 ? 1 : 2;
  static const double block[2][3] = {{0.4, 0.6, 1.1}, {0.6, 1.5, 2.2}}, byte[2][3] = {{0.226, 0.27, 0.4}, {0.25, 0.36, 0.56}};
  return (s.gated ? 2.4 : 1.7) +
         std::max(block[s.gated][tokens] * f8_ceil_div(f8_ceil_div(s.K, kF8Block), 8), byte[s.gated][tokens] * f8_weights(s) - 1);
}

// ------------------------------------------------------------------ a batch
struct F8MidPlan {
  int down, rows, split;  // tiles of x's rows, of so many each; CTAs that share a tile's columns
  double us;
};
constexpr int kMidMaxDown = 65535;  // a tile of x's rows is a grid's y

// How x's rows are cut into tiles and columns into shares, and the microseconds that it takes by the estimate that fits what was
// measured: a CTA's blocks of 128 columns one after the other, or W's bytes, the shares' sums, 4 us for every wave of CTAs behind
// the first; more than 14 clusters of eight are not all there at once. Few tiles of W leave SMs idle with all rows in one tile of x; cut in several, W is read again, from L2, and
// the sums are shorter (256 x 4096 x 1024: 4.9 us in four tiles, 7.7 in one; gated 128 x 2 * 1024 x 4096: 7.2 in four, 9.8).
inline F8MidPlan f8_mid_plan(const F8Size& s, int sms) {
  const int blocks = f8_ceil_div(s.K, kF8Block), least = f8_ceil_div(s.M, s.gated ? 128 : 256);
  const int64_t across = f8_ceil_div(s.N, 128);
  F8MidPlan best = {};
  for (int times : {1, 2, 3, 4, 6, 8}) {
    if (times > 1 && (16 * (times * least - 1) >= s.M || s.M > 2048)) break;
    F8MidPlan q = {};
    q.rows = f8_ceil_div(f8_ceil_div(s.M, times * least), 16) * 16;
    q.down = f8_ceil_div(s.M, q.rows);  // fewer than asked for where the rows of a tile were rounded up
    for (q.split = 8; q.split > 1 && (2 * q.split > blocks || across * q.down * q.split > sms * 7 / 8);) q.split >>= 1;
    const double block = s.gated ? 0.46 + 0.0021 * q.rows : 0.22 + 0.00105 * q.rows;
    const double waves = (double)f8_ceil_div(across * q.down * q.split, sms);
    q.us = 3.1 + 4 * (waves - 1) + std::max(waves * f8_ceil_div(blocks, q.split) * block, f8_weights(s) / 6.5) +
           q.rows * (q.split == 1 ? 0.006 : s.gated ? 0.029 : 0.0137) + (q.split == 8 && across * q.down > 14 ? 1 : 0);
    if (q.down > kMidMaxDown) q.us = std::numeric_limits<double>::infinity();  // cannot be launched
    if (times == 1 || q.us < best.us) best = q;
  }
  return best;
}

// ---------------------------------------------------------------- many rows
constexpr int kManyRows = 256, kManyCols = 256;  // of a tile

// Rows of W a tile (not gated) for so many pairs of CTAs: fewer where that keeps more of them busy. A block of a tile takes what its
// operands' bytes take to an SM, 62 a cycle (264 + 1.03 cycles a row; the instructions take 2 a row), and a tile 2000 cycles besides.
// Measured: 512 x 12288 x 4096 24.2 us with 192, 25.4 with 256; 512 x 4096 x 4096 13.5 with 128, 14.9 with 256; where 224 would give 6 %,
// it gives 2 or takes 3 (777 x 4096 x 8192: 24.9 and 25.3; 2048 x 4096 x 1024: 12.3 and 11.9; x is then read more often), so no change for less
// than a twelfth.
inline int f8_many_wide(const F8Size& s, int pairs) {
  const int64_t down = f8_ceil_div(s.M, kManyRows), blocks = f8_ceil_div(s.K, kF8Block);
  int best = kManyCols;
  int64_t least = INT64_MAX;
  for (int wide = kManyCols; wide >= 128; wide -= 32) {
    const int64_t tiles = down * f8_ceil_div(s.N, wide), waves = (tiles + pairs - 1) / pairs;
    const int64_t cost = waves * ((264 + 103 * wide / 100) * blocks + 2000);
    if (cost < least - least / 12) {
      best = wide;
      least = cost;
    }
  }
  return best;
}

// Microseconds: a pair of CTAs' tiles one after the other, or W's bytes.
inline double f8_many_us(const F8Size& s, int sms) {
  const int pairs = std::max(1, sms / 2), wide = s.gated ? 256 : f8_many_wide(s, pairs);
  const int64_t tiles = (int64_t)f8_ceil_div(s.M, kManyRows) * f8_ceil_div(s.N, s.gated ? 128 : wide);
  // its instructions, or its results
  const double tile = std::max((0.14 + 0.00055 * wide) * f8_ceil_div(s.K, kF8Block), s.gated ? 3.2 : 2.4);
  return 5.4 + std::max(tile * (double)f8_ceil_div(tiles, pairs), f8_weights(s) / (s.gated ? 4.4 : 4.8));
}

// ------------------------------------------------------------------- choice
enum class F8Kernel { kFew, kMid, kMany };

inline F8Kernel f8_kernel(const F8Size& s, int sms, const F8MidPlan& mid) {
  if (s.M <= 32 && f8_few_us(s) <= mid.us) return F8Kernel::kFew;
  return mid.us < f8_many_us(s, sms) ? F8Kernel::kMid : F8Kernel::kMany;
}

}  // namespace bgq
