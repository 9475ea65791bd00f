// f8_product.cu — which kernel multiplies two e4m3 matrices.
//
// Three read the same operands and give the same kinds of results:
//   f8_few.cu   few rows, mma.sync, W straight into registers: next to nothing besides W's bytes, which come at 4.4 TB/s;
//   f8_mid.cu   W as the tensor cores' operand of 128 rows, columns split over CTAs: 4 us besides W's bytes at 6.5 TB/s;
//   f8_many.cu  tiles of 256 x 256: 6 us besides, and the most arithmetic a second.
// The rule below goes by sizes alone, by the times that these measured (CUDA graphs of 24 calls over 130 to 300 MB of weights;
// us, N x K, gated: 2 N x K):
//                     rows:     1     8    16    32    64   128   256   512  1024  2048
//   4096 x 4096       few     4.3   4.7   5.9   8.6  16.0
//                     mid     6.2   6.3   6.4   6.6   7.2   8.6  11.4  15.5  18.9
//                     many                          15.4              15.4  16.4  25.5
//   12288 x 4096      few    11.8  12.3  15.0  23.4
//                     mid    11.2  11.3  11.4  11.5  12.1  14.3  19.8
//                     many                                17.2  18.4  27.2  36.7  65.6
//   4096 x 1024       few     3.2   3.3   3.3   3.5   5.9
//                     mid     4.2   4.3   4.4   4.6   5.1   6.2   8.5  10.6
//                     many                    8.2   8.2   8.3   8.3   8.4   8.7  12.5
//   1024 x 4096       few     5.2   5.5   9.0  12.8
//   gated             mid     5.3   5.5   5.8   6.4   8.1  10.6  11.3  12.4  16.3
//                     many                                      14.9  15.1  15.5  16.9
//   12288 x 4096      few    25.2  25.6  37.0  57.3
//   gated             mid    19.2  19.4  19.8  20.7  23.0  27.3  47.8
//                     many                                31.3  30.2  38.6  67.8   122
#include <algorithm>

#include "f8.h"
#include "kernels.h"

namespace bgq {

// Bytes of weights up to which few rows are sooner done without tensor memory.
static double few_most(int rows, bool gated) {
  if (rows > 32) return 0;
  if (gated) return rows <= 8 ? 8e6 : rows <= 16 ? 3e6 : 2e6;
  return rows <= 8 ? 40e6 : rows <= 16 ? 20e6 : 8e6;
}

static int ceil_div(int a, int b) { return (a + b - 1) / b; }

// us of f8_mid.cu: blocks of 128 columns one after the other in a CTA, or W's bytes, and the shares' sums.
static double mid_us(const F8Prod& p, bool gated, double weights) {
  const int blocks = f8_blocks(p.K), down = ceil_div(p.M, gated ? 128 : 256), tiles = ceil_div(p.N, 128) * down;
  const int rows = ceil_div(ceil_div(p.M, down), 16) * 16;
  int split = 8;
  while (split > 1 && (2 * split > blocks || tiles * split > num_sms() * 7 / 8)) split >>= 1;
  const double block = gated ? 0.46 + 0.0021 * rows : 0.22 + 0.00105 * rows;
  const double waves = ceil_div(tiles * split, num_sms());
  return 4 + std::max(waves * ceil_div(blocks, split) * block, weights / 6.5e6) + (split > 1 ? rows * (gated ? 0.029 : 0.0137) : 0);
}

// us of f8_many.cu.
static double many_us(const F8Prod& p, bool gated, double weights) {
  const int tiles = ceil_div(p.M, 256) * ceil_div(p.N, gated ? 128 : 256);
  return 6.1 + std::max(0.28 * f8_blocks(p.K) * ceil_div(tiles, std::max(1, num_sms() / 2)), weights / 4.3e6);
}

cudaError_t launch_f8_product(const F8Prod& p, bool gated, cudaStream_t s) {
  const double weights = (double)p.N * p.K * (gated ? 2 : 1);
  // the tensor maps' boxes are a block of columns wide
  if (p.K < kF8Block || weights <= few_most(p.M, gated)) return launch_f8_few(p, gated, s);
  // beyond these rows a wave of tiles is full either way
  if (p.M <= 2048 && mid_us(p, gated, weights) < many_us(p, gated, weights)) return launch_f8_mid(p, gated, s);
  return launch_f8_many(p, gated, s);
}

}  // namespace bgq
