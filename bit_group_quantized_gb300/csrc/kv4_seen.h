// kv4_seen.h — which tokens a row of attention over the 4-bit cache sees.
// Plain C++, so that the host can check the arithmetic as the kernels run it.
#pragma once

#include "host_device.h"

namespace bgq {

// The first token that a row at position `pos` (negative where a sequence has more rows than tokens) sees: t > pos - window.
// In 64 bits: with a window near 2^31, which says as much as none, the difference does not fit in 32.
BGQ_HOST_DEVICE int kv4_first_seen(int pos, int window) {
  const long long t = (long long)pos - window + 1;
  return window > 0 && t > 0 ? (int)t : 0;
}
// The token behind the last that it sees, of the `held` that the page list has room for; never negative.
BGQ_HOST_DEVICE int kv4_end_seen(int pos, int kv_len, int held, int causal) {
  const int end = causal ? pos + 1 : kv_len;
  return end < 0 ? 0 : end < held ? end : held;
}

}  // namespace bgq
