// kv4.cu — writing keys and values into the 4-bit cache, and reading them back.
//
// One group of 64 columns of a token's head: bias = min, scale =
// bf16((max - min) / 15), code = floor((x - bias)/scale + 1/2). A code is one
// fused multiply-add: (x - bias) * r + 1.5 * 2^23 rounds to a whole number in
// the low bits of the sum, with r = (1/scale)(1 + 2^-22). The small excess sends exact
// halves up whatever way 1/scale was rounded, and moves no value that is more than 2^-18
// of a step away from a half.
//
// Both kernels are bound by memory (2 bytes of bf16 and 0.56 bytes of cache a
// value), and nearly as much by the instructions that place the codes: 15349 rows of 8 heads of 128 written
// and read back in 33.3 us (4.8 TB/s of the 161 MB both move; issue slots 60 % full in the writing half), 78514 tokens
// of 2 heads of 256 read in 36.5 us (5.6 TB/s). Four lanes share a group, 16 values a lane in two 16-byte loads (the
// reductions over a group then cost two shuffles, and the scale's division
// is spread over 16 values); a lane's codes are two words of the group.
#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace bgq {

constexpr int kKvThreads = 256;
// A thread's unit is 16 values of a token's head, of K and of V; a block looks its rows' places up once and takes this many rounds of
// units (15349 rows of 8 heads of 128 written and read back: 1 round 33.6 us, 2 32.1, 4 34.1, the blocks then being few; a read of
// 78514 tokens of 2 heads of 256: 40.8, 36.2, 35.9).
constexpr int kKvRounds = 2;
constexpr int kKvMaxRows = 256;

struct KvGeo {
  int units_row;   // units of a row
  int rb;          // rows of a block
  uint32_t m_row;  // u / units_row == umulhi(u, m_row) for u, units_row below 2^16
  int chunk;       // units of a row that one block takes
};

__host__ inline KvGeo kv_geo(int heads, int d, int rows) {
  KvGeo g;
  g.units_row = heads * (d / 16);
  g.rb = 1;
  while (g.rb < kKvMaxRows && g.rb * 2 * g.units_row <= kKvThreads * kKvRounds && (long long)rows >= 8ll * num_sms() * g.rb) g.rb *= 2;
  g.chunk = g.rb > 1 || g.units_row <= kKvThreads ? g.units_row : kKvThreads;
  g.m_row = (uint32_t)((0x100000000ull + g.units_row - 1) / g.units_row);
  return g;
}

struct KvUnit {
  int row, head, lane;  // row of the block, head, unit inside the head: 16-byte pieces lane % 4 and 4 + lane % 4 of its group
};
template <int D>
__device__ __forceinline__ KvUnit kv_unit(const KvGeo& g, int u, int u0, int per) {
  KvUnit k;
  k.row = g.rb > 1 ? (int)__umulhi((uint32_t)u, g.m_row) : 0;
  const int r = u - k.row * per + u0;
  k.head = r / (D / 16);
  k.lane = r % (D / 16);
  return k;
}

__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Where the block's rows' tokens stand in head 0 of their pages (-1: nowhere), looked up once; head h is h pages' heads on.
__device__ __forceinline__ void kv_rows(const Kv4View& v, int r0, int nr, long long* at) {
  if ((int)threadIdx.x < nr) at[threadIdx.x] = kv4_row_at(v, r0 + threadIdx.x);
  __syncthreads();
}
// 16 bytes that an earlier kernel may have written while this one was there already: not by the read-only path.
__device__ __forceinline__ uint4 kv_load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Two fp32 values in a register pair: one instruction for both.
__device__ __forceinline__ uint64_t kv_pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void kv_split(uint64_t d, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t kv_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t kv_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <int D>
__global__ void __launch_bounds__(kKvThreads) k_kv4_append(const __grid_constant__ bgq_kv4_cache c,
                                                           const __grid_constant__ Kv4View v,
                                                           const __grid_constant__ KvGeo g,
                                                           const uint16_t* k, long long k_stride,
                                                           const uint16_t* val, long long v_stride) {
  __shared__ long long rows[kKvMaxRows];
  pdl_wait();
  pdl_trigger();
  const int r0 = blockIdx.x * g.rb, nr = min(g.rb, v.rows - r0);
  const int u0 = blockIdx.y * g.chunk, per = min(u0 + g.chunk, g.units_row) - u0, total = nr * per;
  bool ready = false;
  // `total` and the strides are multiples of 4, so the four lanes of a group are in or out together
  for (int u = threadIdx.x; u - (int)threadIdx.x < total; u += kKvThreads) {
    const KvUnit ku = kv_unit<D>(g, u, u0, per);
    const int col = ku.head * D + (ku.lane >> 2) * kGroup + (ku.lane & 3) * 8;
    uint4 in[2][2];
    if (u < total) {
      const uint16_t* ks = k + (long long)(r0 + ku.row) * k_stride + col;
      const uint16_t* vs = val + (long long)(r0 + ku.row) * v_stride + col;
      in[0][0] = kv_load16(ks);
      in[0][1] = kv_load16(ks + 32);
      in[1][0] = kv_load16(vs);
      in[1][1] = kv_load16(vs + 32);
    } else {
      in[0][0] = in[0][1] = in[1][0] = in[1][1] = make_uint4(0, 0, 0, 0);
    }
    if (!ready) {
      kv_rows(v, r0, nr, rows);
      ready = true;
    }
    const long long at = u < total ? rows[ku.row] : -1;
    const long long row = (at < 0 ? 0 : at + (long long)ku.head * c.page_size) * (D / kGroup) + (ku.lane >> 2);  // group's pair
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t* w = &in[i][0].x;  // eight words of two values
      uint32_t lo = w[0], hi = w[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        lo = min_nan2(lo, w[j]);
        hi = max_nan2(hi, w[j]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan2(lo, __shfl_xor_sync(kFull, lo, o));
        hi = max_nan2(hi, __shfl_xor_sync(kFull, hi, o));
      }
      lo = min_nan2(lo, lo >> 16 | lo << 16);
      hi = max_nan2(hi, hi >> 16 | hi << 16);
      const float b = bf16lo(lo), range = bf16lo(hi) - b;
      uint16_t s16 = f2bf(__fdiv_rn(range, 15.f)), b16 = (uint16_t)lo;
      float s = bf16f(s16);
      float r = 0.f;
      if (!(s < __int_as_float(0x7f800000))) {  // a NaN or an infinity among the values
        s16 = b16 = 0x7fc0;
      } else if (s < 0x1p-126f) {
        s16 = 0;  // one value, or a range below normal numbers
      } else {
        r = 1.f / s;
        r = fmaf(r, 0x1p-22f, r);
      }
      constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: whole numbers in the low bits
      const uint64_t b2 = kv_pair(-b, -b), r2 = kv_pair(r, r), whole2 = kv_pair(kWhole, kWhole);
      uint32_t q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t acc = 0;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const uint32_t x2 = w[h * 4 + j];
          float c0, c1;
          kv_split(kv_fma2(kv_add2(kv_pair(bf16lo(x2), bf16hi(x2)), b2), r2, whole2), c0, c1);
          acc = acc * 256 + (__float_as_uint(c1) * 16 + __float_as_uint(c0));
        }
        // every code came with the bits of 1.5 * 2^23 in front: their sum over the eight places
        q[h] = acc - 0x4B400000u * 0x11111111u;
      }
      const bool bad = s16 == 0x7fc0;
      if (at >= 0) {
        uint32_t* qd = (i ? c.v_q : c.k_q) + row * 8 + (ku.lane & 3);
        qd[0] = bad ? 0 : q[0];
        qd[4] = bad ? 0 : q[1];
        if ((ku.lane & 3) == 0) reinterpret_cast<uint32_t*>(i ? c.v_sb : c.k_sb)[row] = (uint32_t)s16 | (uint32_t)b16 << 16;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kKvThreads) k_kv4_read(const __grid_constant__ bgq_kv4_cache c,
                                                         const __grid_constant__ Kv4View v,
                                                         const __grid_constant__ KvGeo g, uint16_t* __restrict__ k,
                                                         long long k_stride, uint16_t* __restrict__ val,
                                                         long long v_stride) {
  __shared__ long long rows[kKvMaxRows];
  __shared__ int held[kKvMaxRows];
  pdl_wait();
  pdl_trigger();
  const int r0 = blockIdx.x * g.rb, nr = min(g.rb, v.rows - r0);
  if ((int)threadIdx.x < nr) {  // rows of no sequence are left as they are
    const int row = r0 + threadIdx.x;
    held[threadIdx.x] = v.q_start ? row >= v.q_start[0] && row < v.q_start[v.batch] : row < v.batch;
  }
  kv_rows(v, r0, nr, rows);
  const int u0 = blockIdx.y * g.chunk, per = min(u0 + g.chunk, g.units_row) - u0, total = nr * per;
  for (int u = threadIdx.x; u < total; u += kKvThreads) {
    const KvUnit ku = kv_unit<D>(g, u, u0, per);
    uint32_t q[2][2], sb[2];
    const long long at = rows[ku.row];
    if (at >= 0) {
      const long long row = (at + (long long)ku.head * c.page_size) * (D / kGroup) + (ku.lane >> 2);  // group's pair
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t* qs = (i ? c.v_q : c.k_q) + row * 8 + (ku.lane & 3);
        q[i][0] = __ldcg(qs);
        q[i][1] = __ldcg(qs + 4);
        sb[i] = __ldcg(reinterpret_cast<const uint32_t*>(i ? c.v_sb : c.k_sb) + row);
      }
    } else {
      q[0][0] = q[0][1] = q[1][0] = q[1][1] = sb[0] = sb[1] = 0;
    }
    if (!held[ku.row]) continue;
    const int col = ku.head * D + (ku.lane >> 2) * kGroup + (ku.lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // A code n places up in a word, put under the exponent of 2^23, is the number 2^23 + code * 16^n (n < 5); the rest of the
      // word comes down three places first. One subtraction, then one fused multiply-add with the scale / 16^n.
      const float s = bf16lo(sb[i]), b = bf16hi(sb[i]);
      const float s1 = s * 0x1p-4f, s2 = s * 0x1p-8f, s3 = s * 0x1p-12f, s4 = s * 0x1p-16f;
      const uint64_t f01 = kv_pair(s, s1), f23 = kv_pair(s2, s3), f42 = kv_pair(s4, s2), f34 = kv_pair(s3, s4);
      const uint64_t b2 = kv_pair(b, b), less = kv_pair(-8388608.f, -8388608.f);
      uint16_t* dst = (i ? val + (long long)(r0 + ku.row) * v_stride : k + (long long)(r0 + ku.row) * k_stride) + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w = q[i][h], wd = w >> 12;
        auto two = [&](uint32_t c0, uint32_t c1, uint64_t f) {
          float v0, v1;
          kv_split(kv_fma2(kv_add2(kv_pair(__uint_as_float(c0 | 0x4B000000u), __uint_as_float(c1 | 0x4B000000u)), less), f, b2), v0, v1);
          const __nv_bfloat162 p2 = __floats2bfloat162_rn(v0, v1);
          return *reinterpret_cast<const uint32_t*>(&p2);
        };
        *reinterpret_cast<uint4*>(dst + h * 32) = make_uint4(two(w & 0xFu, w & 0xF0u, f01), two(w & 0xF00u, w & 0xF000u, f23),
                                                             two(w & 0xF0000u, wd & 0xF00u, f42), two(wd & 0xF000u, wd & 0xF0000u, f34));
      }
    }
  }
}

template <typename... KArgs, typename... Args>
static cudaError_t kv_launch(void (*kern)(KArgs...), const KvGeo& g, int rows, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)rows + g.rb - 1) / g.rb), (g.units_row + g.chunk - 1) / g.chunk);
  cfg.blockDim = dim3(kKvThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

cudaError_t launch_kv4_append(const bgq_kv4_cache& c, const Kv4View& v, const uint16_t* k, long long k_stride,
                              const uint16_t* val, long long v_stride, cudaStream_t s) {
  const KvGeo g = kv_geo(c.kv_heads, c.head_dim, v.rows);
  return kv_launch(c.head_dim == 64 ? k_kv4_append<64> : c.head_dim == 128 ? k_kv4_append<128> : k_kv4_append<256>, g, v.rows, s, c, v, g, k, k_stride, val, v_stride);
}
cudaError_t launch_kv4_read(const bgq_kv4_cache& c, const Kv4View& v, uint16_t* k, long long k_stride, uint16_t* val,
                            long long v_stride, cudaStream_t s) {
  const KvGeo g = kv_geo(c.kv_heads, c.head_dim, v.rows);
  return kv_launch(c.head_dim == 64 ? k_kv4_read<64> : c.head_dim == 128 ? k_kv4_read<128> : k_kv4_read<256>, g, v.rows, s, c, v, g, k, k_stride, val, v_stride);
}

}  // namespace bgq
