// kv4_attn.cu — which kernels an attention call over the 4-bit cache runs.
#include <climits>

#include "attn.h"

namespace bgq {

size_t attn_workspace_bytes(int batch, int rows, int max_q, int q_heads, int kv_heads, int head_dim) {
  return split_workspace_bytes(max_q, q_heads, kv_heads, head_dim);
}

cudaError_t launch_attn(AttnArgs a, cudaStream_t s) {
  a.split_cols = LLONG_MAX;
  return launch_attn_split(a, s);
}

}  // namespace bgq
