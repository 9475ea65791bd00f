// f8_rule.h — which kernel multiplies two e4m3 matrices, and how it cuts them, by sizes alone.
// Plain C++, so that the host can check the arithmetic as the launches run it, and a test can name the kernel that it means.
//
// Three read the same operands and give the same kinds of results:
//   f8_few.cu   few rows, mma.sync, W straight into registers: next to nothing besides W's bytes, which come at 4.4 TB/s;
//   f8_mid.cu   W as the tensor cores' operand of 128 rows, columns split over CTAs: 3 us besides W's bytes at 6.5 TB/s;
//   f8_many.cu  tiles of 256 x 256: 5 us besides, and the most arithmetic a second.
// The one that the estimates call soonest. Measured (CUDA graphs of 24 calls or more, each over weights of its own, 260 MB together,
// us; N x K, gated: 2 N x K):
//                     rows:     1     8    16    32    64   128   256   512  1024  2048  8192
//   4096 x 4096       few      5.1   5.0   6.1   8.7
//                     mid      6.0   6.0   6.1   6.4   7.0   8.0  11.0  14.8  17.8
//                     many                      12.3  12.3  12.8  12.9  13.5  16.4  25.2  81.6
//   12288 x 4096      few     11.4  11.8  14.6  23.0
//                     mid     10.8  10.8  10.9  11.0  11.5  13.5  19.1  35.2  55.6
//                     many                      14.6  16.3  16.6  15.5  23.9  35.8  66.2   254
//   4096 x 1024       few      3.5   3.6   3.2   3.5
//                     mid      3.8   3.9   4.0   4.2   4.5   5.3   5.0   6.3   9.2
//                     many                       7.8   8.2   8.5   6.7   7.1   9.1  13.2  30.7
//   1024 x 1024       few      2.5   2.6   2.1   2.5
//                     mid      3.0   3.1   3.2   3.2   3.6   3.8   4.3   5.0   4.9
//                     many                       5.9   5.9   6.1   6.1   6.1   6.1   6.5  11.8
//   256 x 16384       few      8.5   9.2  11.7  20.2
//                     mid      6.3   6.6   6.6   6.7   6.7   7.0   7.4   8.9  12.7
//                     many                      34.9  35.5  37.0  37.2  37.1  37.0  37.0  40.0
//   1024 x 4096       few      2.9   3.2   3.9   6.2
//                     mid      4.1   4.2   4.3   4.6   5.3   5.2   5.8   7.0  10.0
//                     many                      11.8  11.8  12.3  12.4  12.4  12.6  13.2  25.0
//   1024 x 4096       few      5.2   5.5   9.3  12.6
//   gated             mid      5.2   5.4   5.6   6.2   6.9   7.3   9.2  11.7  15.7
//                     many                      14.8  14.9  15.2  15.3  15.5  16.0  17.8  46.7
//   512 x 1024        few      3.0   3.0   4.1   5.4
//   gated             mid      3.5   3.7   3.9   3.8   3.8   4.3   5.0   5.4   7.1
//                     many                       8.1   8.2   8.3   8.4   8.4   8.4   8.7  13.5
//   12288 x 4096      few     25.0  25.5  37.2  57.0
//   gated             mid     18.1  18.3  18.6  19.4  21.8  25.8  46.9  71.9   142
//                     many                      28.4  28.4  28.8  29.4  38.9  69.6   129   546
// Of these sizes the estimates take the fastest kernel or one within 0.3 us of it. Where no two kernels come
// near each other they may be short, for many rows most: 8192 x 4096 x 1024 22 us (a tile's end lasts longer than its few
// instructions), 8192 x 12288 x 4096 194 (the clock follows the power).
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
  int down, rows, split;  // tiles of x's rows, of so many each; CTAs that share a tile's columns, at most
  double us;
};
constexpr int kMidMaxDown = 65535;  // a tile of x's rows is a grid's y

// How x's rows are cut into tiles and columns into shares, and the microseconds that it takes by the estimate that fits what was
// measured: a CTA's blocks of 128 columns one after the other, or W's bytes, the shares' sums, 4 us for every wave of CTAs behind
// the first. A launch takes half the shares as long as not all of its clusters are there at once (f8_mid.cu; 36 of four, 14 or 15 of eight were);
// the estimate's extra microsecond beyond 14 clusters of eight stands for that, and was fitted with it (gated 64 x 2 * 1024 x 4096, planned
// as 16 of eight, runs as 16 of four). Few tiles of W leave SMs idle with all rows in one tile of x; cut in several, W is read again, from L2,
// and the sums are shorter (256 x 4096 x 1024: 5.0 us in four tiles, 7.7 in one; gated 128 x 2 * 1024 x 4096: 7.3 in four, 9.8).
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
