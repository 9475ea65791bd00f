// kv4_attn.cu — which kernel an attention call over the 4-bit cache runs.
#include "attn.h"
#include "kernels.h"

namespace bgq {

// Columns (query rows times the query heads that share a key head) of the longest sequence up to which kv4_split.cu is
// taken: it takes the cache apart once for every 16 columns, kv4_prompt.cu once for every 128 or 256, but with two
// kernels more and tiles that are always that high. Split and prompt kernel in us, for 24 sequences of 700 to 9000 tokens /
// 100 of 300 to 6000 / one of 65536, eight key heads (the one, and all of 48 columns: two):
//               16 columns                          32 columns                          48 columns
//   head dim 64  32, 62 / 66, 146 / 22, 30           48, 62 / 116, 148 / 22, 30          27, 29 / 51, 50
//           128  45, 76 / 107, 187 / 25, 34          74, 78 / 197, 189 / 31, 33          36, 33 / 78, 59
//           256  95, 111 / 220, 265 / 40, 42         157, 111 / 412, 268 / 53, 42        68, 41 / 169, 86
// (caches still in L2; both kernels are 2 to 4 % slower since they hold values of any sizes. Read from memory, 16 columns of head dim
// 128 take 58, 82 / 130, 194 / 47, 69, and 32 columns 96, 82 / 240, 196 / 76, 69.)
// Where the page lists have room for few tokens (four tiles a warp) and an SM takes one unit of 16 columns at most, the split
// kernel does with one short round what the other does in three launches: 16 sequences of 500 tokens, 40 columns, two key heads:
// 9, 19 us with head dim 64, 12, 22 with 128, 17, 27 with 256; with 128 columns, two units an SM: 22, 20, 28, 24, 44, 29.
static bool few_rows(const bgq_kv4_cache& c, const bgq_kv4_seqs& s, int q_heads) {
  const long long cols = (long long)s.max_q * (q_heads / c.kv_heads);
  if (cols <= (c.head_dim == 256 ? 16 : 32)) return true;
  const long long room = (long long)(s.pages ? s.max_pages : 1) * c.page_size;
  return room <= (c.head_dim == 256 ? 512 : 1024) && (cols + 15) / 16 * s.batch * c.kv_heads <= num_sms();
}

size_t attn_workspace_bytes(const bgq_kv4_cache& c, const bgq_kv4_seqs& s, int q_heads) {
  return few_rows(c, s, q_heads) ? split_workspace_bytes(s.batch, s.max_q, q_heads, c.kv_heads, c.head_dim)
                                 : prompt_workspace_bytes(s.batch, s.rows, q_heads, c.kv_heads, c.head_dim);
}

cudaError_t launch_attn(const AttnArgs& a, const bgq_kv4_seqs& s, cudaStream_t stream) {
  return few_rows(a.c, s, a.q_heads) ? launch_attn_split(a, stream) : launch_attn_prompt(a, stream);
}

}  // namespace bgq
