// f8_product.cu — which kernel multiplies two e4m3 matrices.
//
// Three read the same operands and give the same kinds of results:
//   f8_few.cu   few rows, mma.sync, W straight into registers: next to nothing besides W's bytes, which come at 4.4 TB/s;
//   f8_mid.cu   W as the tensor cores' operand of 128 rows, columns split over CTAs: 3 us besides W's bytes at 6.5 TB/s;
//   f8_many.cu  tiles of 256 x 256: 5 us besides, and the most arithmetic a second.
// The rule below goes by sizes alone: the one that the estimates call soonest. Measured (CUDA graphs of 24 calls over 130 to 300 MB of
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
#include <algorithm>

#include "f8.h"
#include "kernels.h"

namespace bgq {

static int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Microseconds of each kernel; `weights` in millions of bytes.
// Few rows: a warp's blocks of columns one after the other, or W's bytes.
static double few_us(const F8Prod& p, bool gated, double weights) {
  const int tokens = p.M <= 8 ? 0 : p.M <= 16 ? 1 : 2;
  static const double block[2][3] = {{0.4, 0.6, 1.1}, {0.6, 1.5, 2.2}}, byte[2][3] = {{0.226, 0.27, 0.4}, {0.25, 0.36, 0.56}};
  return (gated ? 2.4 : 1.7) + std::max(block[gated][tokens] * ceil_div(f8_blocks(p.K), 8), byte[gated][tokens] * weights - 1);
}

// Many rows: a pair of CTAs' tiles one after the other, or W's bytes.
static double many_us(const F8Prod& p, bool gated, double weights, int sms) {
  const int pairs = std::max(1, sms / 2), wide = gated ? 256 : f8_many_wide(p, pairs);
  const int tiles = ceil_div(p.M, 256) * ceil_div(p.N, gated ? 128 : wide);
  const double tile = std::max((0.14 + 0.00055 * wide) * f8_blocks(p.K), gated ? 3.2 : 2.4);  // its instructions, or its results
  return 5.4 + std::max(tile * ceil_div(tiles, pairs), weights / (gated ? 4.4 : 4.8));
}

cudaError_t launch_f8_product(const F8Prod& p, bool gated, cudaStream_t s) {
  const double weights = (double)p.N * p.K * (gated ? 2e-6 : 1e-6);
  const int sms = num_sms();
  const F8MidPlan mid = f8_mid_plan(p, gated, sms);
  if (p.M <= 32 && few_us(p, gated, weights) <= mid.us) return launch_f8_few(p, gated, s);
  return mid.us < many_us(p, gated, weights, sms) ? launch_f8_mid(p, gated, mid, s) : launch_f8_many(p, gated, s);
}

}  // namespace bgq
