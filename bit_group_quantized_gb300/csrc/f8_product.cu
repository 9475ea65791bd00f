// f8_product.cu — a product of e4m3 matrices by the kernel that f8_rule.h names.
#include "f8.h"
#include "kernels.h"

namespace bgq {

cudaError_t launch_f8_product(const F8Prod& p, bool gated, cudaStream_t s) {
  const F8Size size = {p.M, p.N, p.K, gated};
  const int sms = num_sms();
  const F8MidPlan mid = f8_mid_plan(size, sms);
  switch (f8_kernel(size, sms, mid)) {
    case F8Kernel::kFew: return launch_f8_few(p, gated, s);
    case F8Kernel::kMid: return launch_f8_mid(p, gated, mid, s);
    default: return launch_f8_many(p, gated, s);
  }
}

}  // namespace bgq
