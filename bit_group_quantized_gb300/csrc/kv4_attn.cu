// kv4_attn.cu — attention of grouped query heads over the 4-bit cache.
//
// One warp per row and query head: a lane takes one token of 32, q stays in
// shared memory, the running maximum and sum of the softmax and the output
// stay in registers (lane l holds columns l, l + 32, ...). Per group of 64
// columns q . k = scale * sum(q * code) + bias * sum(q).
#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace bgq {

constexpr int kAttnWarps = 4;

template <int D>
__global__ void __launch_bounds__(kAttnWarps * 32) k_attn(const __grid_constant__ AttnArgs a) {
  constexpr int G = D / kGroup, PL = D / 32;
  __shared__ float qs[kAttnWarps][D];
  __shared__ int s_b;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x, h = blockIdx.y * kAttnWarps + warp;
  if (threadIdx.x == 0) {
    int b = row;
    if (a.v.q_start) {
      int lo = 0, hi = a.v.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.v.q_start[mid] <= row) lo = mid; else hi = mid;
      }
      b = lo;
      if (row < a.v.q_start[b] || row >= a.v.q_start[b + 1]) b = -1;
    }
    s_b = b < a.v.batch ? b : -1;
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0 || h >= a.q_heads) return;
  const Span sp = kv4_span(a.v, b);
  const int pos = sp.kv_len - sp.q_len + (row - sp.first);
  const int end = min(sp.held, a.causal ? pos + 1 : sp.kv_len);
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int kh = h / (a.q_heads / a.c.kv_heads);
  const uint16_t* q = a.q + (long long)row * a.q_stride + h * D;
  for (int i = lane; i < D; i += 32) qs[warp][i] = bf16f(q[i]);
  __syncwarp();
  float qsum[G];
#pragma unroll
  for (int g = 0; g < G; ++g) qsum[g] = warp_sum(qs[warp][g * 64 + lane] + qs[warp][g * 64 + 32 + lane]);
  float m = -INFINITY, l = 0.f, o[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) o[i] = 0.f;
  for (int t0 = begin; t0 < end; t0 += 32) {
    const int t = t0 + lane;
    const int page = t < end ? kv4_page(a.v, b, t) : -1;
    const long long r = page < 0 ? -1 : ((long long)page * a.c.kv_heads + kh) * a.c.page_size + t % a.c.page_size;
    float s = -INFINITY;
    if (r >= 0) {
      s = 0.f;
      const uint32_t* kq = a.c.k_q + r * (D / 8);
      const uint32_t* ks = reinterpret_cast<const uint32_t*>(a.c.k_sb) + r * G;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float acc = 0.f;
        for (int w = 0; w < 8; ++w) {
          const uint32_t c = kq[g * 8 + w];
#pragma unroll
          for (int j = 0; j < 8; ++j) acc = fmaf((float)(c >> (4 * j) & 15u), qs[warp][g * 64 + w * 8 + j], acc);
        }
        s += bf16lo(ks[g]) * acc + bf16hi(ks[g]) * qsum[g];
      }
      s *= a.scale;
    }
    float top = s;  // a NaN score has to reach the sum: kept out of the maximum only
    top = fmaxf(m, warp_max(top));
    const float base = top == -INFINITY ? 0.f : top;
    const float p = r >= 0 ? __expf(s - base) : 0.f, f = __expf(m - base);
    m = top;
    l = l * f + warp_sum(p);
#pragma unroll
    for (int i = 0; i < PL; ++i) o[i] *= f;
    for (int j = 0; j < 32 && t0 + j < end; ++j) {
      const float pj = __shfl_sync(kFull, p, j);
      const long long rj = __shfl_sync(kFull, r, j);
      if (rj < 0) continue;
      const uint32_t* vq = a.c.v_q + rj * (D / 8);
      const uint32_t* vs = reinterpret_cast<const uint32_t*>(a.c.v_sb) + rj * G;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int col = i * 32 + lane;
        const uint32_t code = vq[col >> 3] >> (4 * (col & 7)) & 15u;
        o[i] = fmaf(pj, fmaf((float)code, bf16lo(vs[col >> 6]), bf16hi(vs[col >> 6])), o[i]);
      }
    }
  }
  const bool none = l == 0.f;
  uint16_t* out = a.out + (long long)row * a.out_stride + h * D;
#pragma unroll
  for (int i = 0; i < PL; ++i) out[i * 32 + lane] = f2bf(none ? 0.f : o[i] / l);
  if (a.lse && lane == 0) a.lse[(long long)row * a.q_heads + h] = none ? -INFINITY : m + logf(l);
}

size_t attn_workspace_bytes(int batch, int rows, int max_q, int q_heads, int kv_heads, int head_dim) { return 256; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.v.rows, (a.q_heads + kAttnWarps - 1) / kAttnWarps);
  cfg.blockDim = dim3(kAttnWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a.c.head_dim == 64 ? k_attn<64> : a.c.head_dim == 128 ? k_attn<128> : k_attn<256>, a);
}

}  // namespace bgq
