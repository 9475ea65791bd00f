// f8_product.cu — which kernel multiplies two e4m3 matrices.
#include "f8.h"

namespace bgq {

cudaError_t launch_f8_product(const F8Prod& p, bool gated, cudaStream_t s) {
  // the tensor maps' boxes are a block of columns wide
  if (p.M <= 32 || p.K < kF8Block) return launch_f8_few(p, gated, s);
  return p.M <= 512 ? launch_f8_mid(p, gated, s) : launch_f8_many(p, gated, s);
}

}  // namespace bgq
