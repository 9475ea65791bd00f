// kv4_attn.cu — which kernel an attention call over the 4-bit cache runs.
#include "attn.h"

namespace bgq {

// Columns (query rows times the query heads that share a key head) of the longest sequence up to which kv4_split.cu is
// taken: it takes the cache apart once for every 16 columns, kv4_prompt.cu once for every 128 or 256, but with two
// kernels more and tiles that are always that high. Split and prompt kernel in us, for 24 sequences of 700 to 9000 tokens /
// 100 of 300 to 6000 / one of 65536, eight key heads (the one, and all of 48 columns: two):
//               16 columns                          32 columns                          48 columns
//   head dim 64  32, 62 / 66, 146 / 22, 30           48, 62 / 116, 148 / 22, 30          27, 29 / 51, 50
//           128  45, 76 / 107, 187 / 25, 34          74, 78 / 197, 189 / 31, 33          36, 33 / 78, 59
//           256  95, 111 / 220, 265 / 40, 42         157, 111 / 412, 268 / 53, 42        68, 41 / 169, 86
static bool few_rows(int max_q, int q_heads, int kv_heads, int head_dim) {
  return (long long)max_q * (q_heads / kv_heads) <= (head_dim == 256 ? 16 : 32);
}

size_t attn_workspace_bytes(int batch, int rows, int max_q, int q_heads, int kv_heads, int head_dim) {
  return few_rows(max_q, q_heads, kv_heads, head_dim) ? split_workspace_bytes(batch, max_q, q_heads, kv_heads, head_dim)
                                                      : prompt_workspace_bytes(batch, rows, q_heads, kv_heads, head_dim);
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
  return few_rows(a.max_q, a.q_heads, a.c.kv_heads, a.c.head_dim) ? launch_attn_split(a, s) : launch_attn_prompt(a, s);
}

}  // namespace bgq
