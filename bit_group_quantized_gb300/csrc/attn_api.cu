// attn_api.cu — the attention entry points of the C ABI (include/bgq.h):
// argument checks, then the launches of rope.cu, kv4.cu and kv4_attn.cu.
#include <math.h>
#include <string.h>

#include "attn.h"

using namespace bgq;

namespace {

constexpr int kMaxHeads = 256;
constexpr int kMaxSeqs = 4096;
constexpr int64_t kMaxTokens = INT32_MAX - 65535;  // of a sequence: kernels step past the last by less than the rest

inline bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline cudaStream_t st(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? BGQ_OK : BGQ_ERR_CUDA; }

// A strided array of rows of `width` bf16 values, read and written in 16-byte pieces.
int check_rows(const void* p, int64_t stride, int64_t width) {
  if (!p || !al(p, 16) || stride < width || stride % 8) return BGQ_ERR_INVALID_ARG;
  return BGQ_OK;
}

int check_cache(const bgq_kv4_cache* c) {
  if (!c || !c->k_q || !c->k_sb || !c->v_q || !c->v_sb) return BGQ_ERR_INVALID_ARG;
  if (!al(c->k_q, 16) || !al(c->k_sb, 16) || !al(c->v_q, 16) || !al(c->v_sb, 16)) return BGQ_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 16 || c->page_size % 16 || c->kv_heads < 1) return BGQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return BGQ_ERR_UNSUPPORTED;
  // kernels count a pool's heads, and 16-token blocks of them, in 32 bits
  if (c->kv_heads > kMaxHeads || (int64_t)c->n_pages * c->kv_heads > INT32_MAX / (c->page_size / 16)) return BGQ_ERR_UNSUPPORTED;
  return BGQ_OK;
}

int check_seqs(const bgq_kv4_seqs* s) {
  if (!s || !s->kv_len || !al(s->kv_len, 4) || !al(s->q_start, 4) || !al(s->pages, 4)) return BGQ_ERR_INVALID_ARG;
  if (s->batch < 1 || s->rows < 0 || s->max_q < 1) return BGQ_ERR_INVALID_ARG;
  if (s->pages && s->max_pages < 1) return BGQ_ERR_INVALID_ARG;
  if (!s->q_start && (s->rows != s->batch || s->max_q != 1)) return BGQ_ERR_INVALID_ARG;
  if (s->batch > kMaxSeqs) return BGQ_ERR_UNSUPPORTED;
  return BGQ_OK;
}

Kv4View view(const bgq_kv4_cache* c, const bgq_kv4_seqs* s) {
  Kv4View v;
  v.q_start = s->q_start;
  v.kv_len = s->kv_len;
  v.pages = s->pages;
  v.batch = s->batch;
  v.max_pages = s->pages ? s->max_pages : 1;
  v.rows = s->rows;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.heads = c->kv_heads;
  v.cap = (long long)v.max_pages * v.page_size;
  if (v.cap > kMaxTokens) v.cap = kMaxTokens;
  return v;
}

int check_plan(const bgq_rope_plan* p) {
  if (!p || p->head_dim < 16 || p->head_dim > 256 || p->head_dim % 8) return BGQ_ERR_INVALID_ARG;
  if (p->rot_dim < 16 || p->rot_dim > p->head_dim || p->rot_dim % 16) return BGQ_ERR_INVALID_ARG;
  if (p->n_axes < 1 || p->n_axes > BGQ_ROPE_MAX_AXES) return BGQ_ERR_INVALID_ARG;
  for (int i = 0; i < p->rot_dim / 2; ++i)
    if (p->axis[i] >= p->n_axes) return BGQ_ERR_INVALID_ARG;
  return BGQ_OK;
}

}  // namespace

extern "C" {

int32_t bgq_rope_init(bgq_rope_plan* p, int32_t head_dim, int32_t rot_dim, double theta, int32_t n_axes,
                      const int32_t* sections, int32_t flags) {
  if (!p || !sections || head_dim < 1 || rot_dim < 1 || rot_dim > head_dim) return BGQ_ERR_INVALID_ARG;
  if (!(theta > 0) || !isfinite(theta) || n_axes < 1) return BGQ_ERR_INVALID_ARG;
  if (flags & ~(BGQ_ROPE_PAIRS | BGQ_ROPE_CYCLE | BGQ_ROPE_RESTART)) return BGQ_ERR_INVALID_ARG;
  if ((flags & BGQ_ROPE_CYCLE) && (flags & BGQ_ROPE_RESTART)) return BGQ_ERR_INVALID_ARG;
  if (head_dim > 256 || head_dim % 8 || head_dim < 16 || rot_dim % 16 || n_axes > BGQ_ROPE_MAX_AXES) return BGQ_ERR_UNSUPPORTED;
  const int half = rot_dim / 2;
  int64_t sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0) return BGQ_ERR_INVALID_ARG;
    sum += sections[a];
  }
  if (sum != half) return BGQ_ERR_INVALID_ARG;
  memset(p, 0, sizeof *p);
  p->head_dim = head_dim;
  p->rot_dim = rot_dim;
  p->n_axes = n_axes;
  p->flags = flags;
  int first = 0;  // first pair of axis a's section
  for (int a = 0; a < n_axes; first += sections[a], ++a)
    for (int i = first; i < first + sections[a]; ++i) p->axis[i] = (uint8_t)a;
  if (flags & BGQ_ROPE_CYCLE)
    for (int i = 0; i < half; ++i) {
      const int a = i % n_axes;
      p->axis[i] = (uint8_t)(i / n_axes < sections[a] ? a : 0);
    }
  first = 0;
  for (int a = 0; a < n_axes; first += sections[a], ++a)
    for (int i = first; i < first + sections[a]; ++i) {
      const double e = (flags & BGQ_ROPE_RESTART) ? (double)(i - first) / sections[a] : (double)i / half;
      const double turns = pow(theta, -e) / 6.283185307179586476925286766559;  // of one position step
      const double part = turns - floor(turns);                                 // whole turns change nothing
      p->freq[i] = part >= 1.0 ? 0 : (uint64_t)(part * 18446744073709551616.0);
    }
  return BGQ_OK;
}

int32_t bgq_rope(const bgq_rope_plan* p, const uint16_t* x, int64_t x_stride, const int32_t* pos, int64_t pos_stride,
                 int32_t tokens, int32_t heads, uint16_t* y, int64_t y_stride, int32_t inverse, void* stream) {
  int r = check_plan(p);
  if (r) return r;
  if (tokens < 0 || heads < 1) return BGQ_ERR_INVALID_ARG;
  if (heads > 1024) return BGQ_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)heads * p->head_dim;
  if ((r = check_rows(x, x_stride, width)) || (r = check_rows(y, y_stride, width))) return r;
  if (!pos || !al(pos, 4) || pos_stride < 0 || (p->n_axes > 1 && pos_stride && pos_stride < tokens)) return BGQ_ERR_INVALID_ARG;
  if (x == y && x_stride != y_stride) return BGQ_ERR_INVALID_ARG;
  if (tokens == 0) return BGQ_OK;
  return cuda_status(launch_rope(*p, x, x_stride, pos, pos_stride, tokens, heads, y, y_stride, inverse != 0, st(stream)));
}

int32_t bgq_kv4_append(const bgq_kv4_cache* c, const bgq_kv4_seqs* s, const uint16_t* k, int64_t k_stride,
                       const uint16_t* v, int64_t v_stride, void* stream) {
  int r = check_cache(c);
  if (r || (r = check_seqs(s))) return r;
  const int64_t width = (int64_t)c->kv_heads * c->head_dim;
  if ((r = check_rows(k, k_stride, width)) || (r = check_rows(v, v_stride, width))) return r;
  if (s->rows == 0) return BGQ_OK;
  return cuda_status(launch_kv4_append(*c, view(c, s), k, k_stride, v, v_stride, st(stream)));
}

int32_t bgq_kv4_read(const bgq_kv4_cache* c, const bgq_kv4_seqs* s, uint16_t* k, int64_t k_stride, uint16_t* v,
                     int64_t v_stride, void* stream) {
  int r = check_cache(c);
  if (r || (r = check_seqs(s))) return r;
  const int64_t width = (int64_t)c->kv_heads * c->head_dim;
  if ((r = check_rows(k, k_stride, width)) || (r = check_rows(v, v_stride, width))) return r;
  if (s->rows == 0) return BGQ_OK;
  return cuda_status(launch_kv4_read(*c, view(c, s), k, k_stride, v, v_stride, st(stream)));
}

static int check_heads(const bgq_kv4_cache* c, int32_t q_heads) {
  if (q_heads < 1 || q_heads % c->kv_heads) return BGQ_ERR_INVALID_ARG;
  if (q_heads / c->kv_heads > 64 || q_heads > 1024) return BGQ_ERR_UNSUPPORTED;
  return BGQ_OK;
}

size_t bgq_kv4_attention_workspace_bytes(const bgq_kv4_cache* c, const bgq_kv4_seqs* s, int32_t q_heads) {
  if (check_cache(c) || check_seqs(s) || check_heads(c, q_heads)) return 0;
  return attn_workspace_bytes(*c, *s, q_heads);
}

int32_t bgq_kv4_attention(const bgq_kv4_cache* c, const bgq_kv4_seqs* s, const uint16_t* q, int64_t q_stride,
                          int32_t q_heads, float scale, int32_t causal, int32_t window, uint16_t* out,
                          int64_t out_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
  int r = check_cache(c);
  if (r || (r = check_seqs(s)) || (r = check_heads(c, q_heads))) return r;
  const int64_t width = (int64_t)q_heads * c->head_dim;
  if ((r = check_rows(q, q_stride, width)) || (r = check_rows(out, out_stride, width))) return r;
  if (!al(lse, 4) || !isfinite(scale) || window < 0) return BGQ_ERR_INVALID_ARG;
  if (!ws || !al(ws, 256) ||
      ws_bytes < attn_workspace_bytes(*c, *s, q_heads))
    return BGQ_ERR_WORKSPACE;
  if ((int64_t)s->rows * (q_heads / c->kv_heads) > kMaxTokens) return BGQ_ERR_UNSUPPORTED;  // kernels round it up to a tile
  if (s->rows == 0) return BGQ_OK;
  AttnArgs a;
  a.c = *c;
  a.v = view(c, s);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.q_heads = q_heads;
  a.causal = causal != 0;
  a.window = window;
  a.max_q = s->max_q;
  a.page_shift = (c->page_size & (c->page_size - 1)) ? -1 : __builtin_ctz(c->page_size);
  a.group = q_heads / c->kv_heads;
  a.group_inv = a.group > 1 ? ~(uint64_t)0 / a.group + 1 : 0;
  a.scale = scale;
  a.ws = ws;
  return cuda_status(launch_attn(a, *s, st(stream)));
}

}  // extern "C"
