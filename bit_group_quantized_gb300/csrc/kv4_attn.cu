// kv4_attn.cu — which kernel an attention call over the 4-bit cache runs.
#include "attn.h"

namespace bgq {

// Columns (query rows times the query heads that share a key head) of the longest sequence: up to
// kSplitCols the call is bound by reading the cache once, which kv4_split.cu does best;
// beyond, kv4_split.cu would take the cache apart once for every 16 columns.
constexpr int kSplitCols = 16;
static bool few_rows(int max_q, int q_heads, int kv_heads) { return (long long)max_q * (q_heads / kv_heads) <= kSplitCols; }

size_t attn_workspace_bytes(int batch, int rows, int max_q, int q_heads, int kv_heads, int head_dim) {
  return few_rows(max_q, q_heads, kv_heads) ? split_workspace_bytes(max_q, q_heads, kv_heads, head_dim)
                                            : prompt_workspace_bytes(batch, rows, q_heads, kv_heads, head_dim);
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
  return few_rows(a.max_q, a.q_heads, a.c.kv_heads) ? launch_attn_split(a, s) : launch_attn_prompt(a, s);
}

}  // namespace bgq
