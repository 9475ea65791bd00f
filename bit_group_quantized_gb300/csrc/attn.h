// attn.h — internal interface between the attention entry points (attn_api.cu)
// and their kernels: rotary positions (rope.cu), the 4-bit cache (kv4.cu) and
// attention over it (kv4_attn.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/bgq.h"

namespace bgq {

// Allows a kernel `bytes` of dynamic shared memory on the current device: asked for once per device and kernel.
template <typename K>
inline cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The sequences of a call as kernels see them. Every length, row and page
// number is read from device memory, so each is checked where it is used:
// rows outside [0, rows), positions outside the sequence and pages outside
// the pool are passed over.
struct Kv4View {
  const int32_t* q_start;  // [batch+1], or null: sequence b has the one row b
  const int32_t* kv_len;   // [batch]
  const int32_t* pages;    // [batch][max_pages], or null: sequence b has the one page b
  int batch, max_pages, rows;
  int n_pages, page_size, heads;
  long long cap;  // tokens a sequence's page list can hold: max_pages * page_size
};

struct Span {  // the rows of one sequence and its tokens
  int first, q_len;
  int kv_len;  // with the rows' own tokens: row j stands at position kv_len - q_len + j
  int held;    // tokens that the page list has room for (kv_len, unless the caller's list is too short)
};

__device__ __forceinline__ Span kv4_span(const Kv4View& v, int b) {
  Span s;
  s.first = v.q_start ? v.q_start[b] : b;
  const int end = v.q_start ? v.q_start[b + 1] : b + 1;
  s.q_len = end > s.first ? (int)min((uint32_t)end - (uint32_t)s.first, 0x7fffffffu) : 0;
  s.kv_len = max(v.kv_len[b], 0);
  s.held = s.kv_len > v.cap ? (int)v.cap : s.kv_len;
  return s;
}

// Pool page that holds token t of sequence b, or -1.
__device__ __forceinline__ int kv4_page(const Kv4View& v, int b, int t) {
  const int p = v.pages ? v.pages[(long long)b * v.max_pages + t / v.page_size] : b;
  return p >= 0 && p < v.n_pages ? p : -1;
}

// Where a row's token stands in head 0 of its page: its row of the pool's [n_pages][heads][page_size], or -1.
__device__ __forceinline__ long long kv4_row_at(const Kv4View& v, int row) {
  int b = row;
  if (v.q_start) {  // the last sequence that starts at or before the row
    int lo = 0, hi = v.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (v.q_start[mid] <= row) lo = mid; else hi = mid;
    }
    b = lo;
    if (row < v.q_start[b] || row >= v.q_start[b + 1]) return -1;
  }
  if (b >= v.batch) return -1;
  const int end = v.q_start ? v.q_start[b + 1] : b + 1;
  const long long t = (long long)v.kv_len[b] - end + row;
  if (t < 0 || t >= v.cap) return -1;
  const int p = kv4_page(v, b, (int)t);
  return p < 0 ? -1 : (long long)p * v.heads * v.page_size + (int)t % v.page_size;
}

cudaError_t launch_rope(const bgq_rope_plan& p, const uint16_t* x, long long x_stride, const int32_t* pos,
                        long long pos_stride, int tokens, int heads, uint16_t* y, long long y_stride, bool inverse,
                        cudaStream_t s);
cudaError_t launch_kv4_append(const bgq_kv4_cache& c, const Kv4View& v, const uint16_t* k, long long k_stride,
                              const uint16_t* val, long long v_stride, cudaStream_t s);
cudaError_t launch_kv4_read(const bgq_kv4_cache& c, const Kv4View& v, uint16_t* k, long long k_stride, uint16_t* val,
                            long long v_stride, cudaStream_t s);

// Bytes at the start of an attention workspace that only the control block and kv4_split.cu's arrival counters use, which
// every call leaves at zero: calls of both kernels and of any shapes may share a workspace.
constexpr int kAttnHead = 4096;

struct AttnArgs {
  bgq_kv4_cache c;
  Kv4View v;
  const uint16_t* q;
  uint16_t* out;
  float* lse;  // nullable
  long long q_stride, out_stride;
  int q_heads, causal, window, max_q;
  int page_shift;  // log2 of the page size, or -1
  int group;       // q_heads / kv_heads
  uint64_t group_inv;  // ceil(2^64 / group), 0 for one head
  float scale;
  void* ws;
};
size_t attn_workspace_bytes(const bgq_kv4_cache& c, const bgq_kv4_seqs& s, int q_heads);
cudaError_t launch_attn(const AttnArgs& a, const bgq_kv4_seqs& s, cudaStream_t stream);

size_t split_workspace_bytes(int batch, int max_q, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_attn_split(const AttnArgs& a, cudaStream_t s);
size_t prompt_workspace_bytes(int batch, int rows, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_attn_prompt(const AttnArgs& a, cudaStream_t s);

}  // namespace bgq
