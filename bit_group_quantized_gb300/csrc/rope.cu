// rope.cu — rotary positions with several axes.
//
// Pair i of a head, (a, b), turns by the angle t = pos[axis(i)] * f_i:
// (a cos t - b sin t, a sin t + b cos t). The plan holds f_i in turns (f_i / 2 pi) as a 64-bit
// fixed-point fraction, off by at most 2^-54 as it comes from a double (theta >= 1). The product pos * f_i modulo 2^64 is exact, so
// the angle is off by |pos| 2^-54 turns (2^-23 at the farthest positions, 2^-34 at a million), and no
// range reduction is left to do. Its upper 32 bits go to sincospi.
//
// Bound by memory (2 bytes in, 2 bytes out per value). A block takes whole
// tokens: its first loads are in flight while it computes the angles of its
// tokens once, for all heads, into shared memory. 8191 tokens of 40 heads of 128: 27.4 us, 6.1 TB/s,
// 92 % of a copy's rate. Few tokens cost what a launch costs (64 tokens: about 7 us a call through Python).
// Sums and products are fp32; the result is rounded to bf16 once.
#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace bgq {

constexpr int kRopeMaxThreads = 512;
constexpr int kRopeLoads = 4;       // units a thread has in flight
constexpr int kRopeMaxTokens = 16;  // tokens of a block

struct RopeGeo {
  int upt;            // units of a head: half/8 pairs of 16-byte chunks, then 16-byte chunks behind rot
  int units_tok;      // units of a token
  uint32_t m_upt, m_tok;  // ceil(2^32 / .): u / n == umulhi(u, m) for u, n below 2^16
  int tb;             // tokens of a block
  int chunk;          // units of a token that one block takes (grid.y blocks share a token)
};

// HALF: pair i is columns (i, i + rot/2): a unit is 8 pairs, two 16-byte chunks.
// Otherwise pair i is columns (2i, 2i+1): a unit is one 16-byte chunk, 4 pairs.
template <bool HALF>
__global__ void __launch_bounds__(kRopeMaxThreads) k_rope(const __grid_constant__ bgq_rope_plan p,
                                                       const __grid_constant__ RopeGeo g, const uint16_t* x, long long x_stride,
                                                       const int32_t* pos,
                                                       long long pos_stride, int tokens, uint16_t* y,
                                                       long long y_stride, float sign) {
  // cos and sin of two pairs side by side, [tb][pairs of a unit / 2][units of a head]: threads on neighbouring units read
  // neighbouring 16 bytes
  extern __shared__ __align__(16) float4 cs[];
  constexpr int kPair = HALF ? 8 : 4;  // pairs of a unit
  pdl_wait();
  pdl_trigger();
  const int half = p.rot_dim >> 1;
  const int turn_units = HALF ? half >> 3 : p.rot_dim >> 3;
  const int t0 = blockIdx.x * g.tb, nt = min(g.tb, tokens - t0);
  const int u0 = blockIdx.y * g.chunk, u1 = min(u0 + g.chunk, g.units_tok);
  const int per = u1 - u0, total = nt * per;

  auto place = [&](int u, int& tok, int& col, int& unit) {
    tok = g.tb == 1 ? 0 : per == 1 ? u : (int)__umulhi((uint32_t)u, g.m_tok);  // several tokens: whole ones
    const int r = u - tok * per + u0;
    const int head = g.upt > 1 ? (int)__umulhi((uint32_t)r, g.m_upt) : r;
    unit = r - head * g.upt;
    col = head * p.head_dim + (unit < turn_units ? unit * 8 : p.rot_dim + (unit - turn_units) * 8);
  };
  bool ready = false;
  const int T = blockDim.x;
  for (int base = threadIdx.x; base - (int)threadIdx.x < total; base += T * kRopeLoads) {
    uint4 lo[kRopeLoads], hi[kRopeLoads];
#pragma unroll
    for (int k = 0; k < kRopeLoads; ++k) {
      const int u = base + k * T;
      if (u < total) {
        int tok, col, unit;
        place(u, tok, col, unit);
        const uint16_t* s = x + (long long)(t0 + tok) * x_stride + col;
        lo[k] = *reinterpret_cast<const uint4*>(s);
        if (HALF && unit < turn_units) hi[k] = *reinterpret_cast<const uint4*>(s + half);
      }
    }
    if (!ready) {
      for (int i = threadIdx.x; i < nt * half; i += T) {
        const int tok = i / half, pr = i - tok * half;
        const long long at = pos[p.axis[pr] * pos_stride + t0 + tok];
        const unsigned long long turn = (unsigned long long)at * p.freq[pr];
        float s, c;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);  // [-1, 1) half turns
        const int un = pr / kPair, in = pr % kPair;
        reinterpret_cast<float2*>(cs + (tok * (kPair / 2) + in / 2) * turn_units + un)[in & 1] = make_float2(c, s * sign);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < kRopeLoads; ++k) {
      const int u = base + k * T;
      if (u < total) {
        int tok, col, unit;
        place(u, tok, col, unit);
        uint16_t* o = y + (long long)(t0 + tok) * y_stride + col;
        if (unit < turn_units) {
          uint32_t* l = &lo[k].x;
          if (HALF) {
            uint32_t* h = &hi[k].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 c = cs[(tok * 4 + j) * turn_units + unit];
              const float a0 = bf16lo(l[j]), a1 = bf16hi(l[j]), b0 = bf16lo(h[j]), b1 = bf16hi(h[j]);
              const __nv_bfloat162 lv = __floats2bfloat162_rn(fmaf(a0, c.x, -b0 * c.y), fmaf(a1, c.z, -b1 * c.w));
              const __nv_bfloat162 hv = __floats2bfloat162_rn(fmaf(a0, c.y, b0 * c.x), fmaf(a1, c.w, b1 * c.z));
              l[j] = *reinterpret_cast<const uint32_t*>(&lv);
              h[j] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            *reinterpret_cast<uint4*>(o + half) = hi[k];
          } else {
            const float4 c4[2] = {cs[tok * 2 * turn_units + unit], cs[(tok * 2 + 1) * turn_units + unit]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 c = j & 1 ? make_float2(c4[j >> 1].z, c4[j >> 1].w) : make_float2(c4[j >> 1].x, c4[j >> 1].y);
              const float a = bf16lo(l[j]), b = bf16hi(l[j]);
              const __nv_bfloat162 v = __floats2bfloat162_rn(fmaf(a, c.x, -b * c.y), fmaf(a, c.y, b * c.x));
              l[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
          }
        }
        *reinterpret_cast<uint4*>(o) = lo[k];
      }
    }
  }
}

cudaError_t launch_rope(const bgq_rope_plan& p, const uint16_t* x, long long x_stride, const int32_t* pos,
                        long long pos_stride, int tokens, int heads, uint16_t* y, long long y_stride, bool inverse,
                        cudaStream_t s) {
  const bool pairs = p.flags & BGQ_ROPE_PAIRS;
  const int half = p.rot_dim / 2;
  RopeGeo g;
  g.upt = (pairs ? p.rot_dim : half) / 8 + (p.head_dim - p.rot_dim) / 8;
  g.units_tok = g.upt * heads;
  // A block takes as many tokens as fill its threads' loads (up to 384 threads, which leaves an SM its five blocks), unless
  // that leaves SMs without a block; a token of many heads is shared out. The threads divide the units evenly: with a
  // fixed 256 the 320 units of 40 heads of 128 left most of them idle (8191 tokens: 36 us).
  const int most = 384 * kRopeLoads;
  g.tb = 1;
  while (g.tb < kRopeMaxTokens && g.tb * 2 * g.units_tok <= most && (long long)tokens >= 4ll * num_sms() * g.tb) g.tb *= 2;
  g.chunk = g.tb > 1 || g.units_tok <= most ? g.units_tok : most;
  const int loads = tokens < num_sms() * 4 ? 1 : kRopeLoads;  // few tokens: more threads, fewer units each
  const int threads = std::min(kRopeMaxThreads, ((g.tb * g.chunk + loads - 1) / loads + 31) / 32 * 32);
  g.m_upt = (uint32_t)((0x100000000ull + g.upt - 1) / g.upt);
  g.m_tok = (uint32_t)((0x100000000ull + g.units_tok - 1) / g.units_tok);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)tokens + g.tb - 1) / g.tb), (g.units_tok + g.chunk - 1) / g.chunk);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)g.tb * half * sizeof(float2);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pairs ? k_rope<false> : k_rope<true>, p, g, x, x_stride, pos, pos_stride, tokens, y,
                            y_stride, inverse ? -1.f : 1.f);
}

}  // namespace bgq
