// f8_few.cu — products of e4m3 matrices for few rows: one pass over the weights.
//
// A CTA takes 16 rows of W (gated: 16 of gate and the same of up) and up to 8 NT rows of x. Its eight warps share the blocks of
// 128 columns; in a block a warp reads W straight into the fragments of mma.sync m16n8k32: lane (g, t) has 16 columns
// in one load, of rows g and g + 8, which serve two matrix instructions (the columns of a step may be any, as long as
// both operands take the same). A block's sum (four steps, each cut to fp32) is scaled and added in fp32; the warps' sums meet in shared
// memory and are added in warp order. What bounds it: loads in flight, two CTAs an SM with 128 registers a thread, which
// bring W at 4.4 TB/s (1 row, 12288 x 4096: 11.4 us; 4096 x 4096: 5.1). Four CTAs with half the loads each: 13.8 us; 32-byte loads: 12.7;
// pieces of rows by bulk copies to shared memory: 12.8. W's lines are asked into L2 while the kernel before still runs (without: 5.6 us
// where it was 4.3 then).
//
// Gated with an e4m3 result: a block of 128 columns of the result is the work of 8 CTAs, one cluster, which exchange
// their rows' largest magnitudes.
#include "common.cuh"
#include "f8.h"
#include "kernels.h"
#include "tc.cuh"

namespace bgq {

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32, kFewPitch = 20;
constexpr int kFewCluster = kF8Block / 16;

__device__ __forceinline__ void f8_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 2^e for -127 <= e <= 127. 2^-127 as 0: it is half of a scale of 2^-253 or 2^-254 then, and a block's sum, below 2^25, is far below
// fp32's range behind it.
__device__ __forceinline__ float f8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint4 f8_ld_weights(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Blocks a warp loads before it multiplies them: what its registers hold (17 to 32 rows, gated, spill 268 bytes all the same; few sizes take that).
template <int NT, bool GATED>
constexpr int few_ahead() { return NT == 1 ? (GATED ? 2 : 4) : NT == 2 ? (GATED ? 1 : 2) : 1; }

template <int NT, bool GATED>
__global__ void __launch_bounds__(kFewThreads, 2) k_f8_few(const F8Prod p) {
  constexpr int R = GATED ? 2 : 1, T = 8 * NT, U = few_ahead<NT, GATED>();
  __shared__ __align__(16) float part[kFewWarps][R][T][kFewPitch];
  __shared__ uint32_t most[T];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int blocks = f8_blocks(p.K);
  // W into L2 while the kernel before this one ends (L2 holds whatever is written there in the meantime)
#pragma unroll
  for (int r = 0; r < R; ++r)
    for (int i = tid; i < 16 * blocks; i += kFewThreads) {
      const int row = n0 + (i & 15), col = (i >> 4) * kF8Block;
      if (row < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w[r] + row * p.w_stride[r] + col));
    }
  pdl_wait();
  pdl_trigger();
  float sum[R][NT][4] = {};
  for (int first = warp; first < blocks; first += kFewWarps * U) {
    uint4 w[U][R][2][2], x[U][NT][2];  // [.][.][half of the block][row g or g + 8]
    int ew[U][R], ex[U][NT][2];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int kb = first + k * kFewWarps, c0 = kb * kF8Block + t * 16;  // past the last block nothing is loaded
      const bool there = kb < blocks;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = c0 + half * 64, row = n0 + g + 8 * i;
            w[k][r][half][i] = make_uint4(0, 0, 0, 0);
            if (row < p.N && col < p.K) w[k][r][half][i] = f8_ld_weights(p.w[r] + row * p.w_stride[r] + col);
          }
        ew[k][r] = there && n0 < p.N ? p.ws[r][(int64_t)(n0 / kF8Block) * p.ws_stride[r] + kb] : 0;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int col = c0 + half * 64, row = 8 * j + g;
          x[k][j][half] = make_uint4(0, 0, 0, 0);
          if (row < p.M && col < p.K) x[k][j][half] = *reinterpret_cast<const uint4*>(p.x + row * p.x_stride + col);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * j + 2 * t + i;
          ex[k][j][i] = there && row < p.M ? p.xs[row * p.xs_stride + kb] : 0;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 &w0 = w[k][r][half][0], &w1 = w[k][r][half][1], &b = x[k][j][half];
            f8_mma(d, w0.x, w1.x, w0.y, w1.y, b.x, b.y);
            f8_mma(d, w0.z, w1.z, w0.w, w1.w, b.z, b.w);
          }
          // times 2^(ew + ex - 254) in two halves, neither of which leaves fp32's range unless the result does
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int e = ew[k][r] + ex[k][j][i] - 254, lo = e >> 1;
            const float f0 = f8_pow2(lo), f1 = f8_pow2(e - lo);
            sum[r][j][i] = fmaf(d[i] * f0, f1, sum[r][j][i]);
            sum[r][j][i + 2] = fmaf(d[i + 2] * f0, f1, sum[r][j][i + 2]);
          }
        }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][r][8 * j + 2 * t + (i & 1)][g + 8 * (i >> 1)] = sum[r][j][i];
  __syncthreads();
  // a thread has row n = tid % 16 of W and the rows tid / 16, 16 more on, ... of x
  const int n = tid & 15;
  constexpr int kEach = (T * 16 + kFewThreads - 1) / kFewThreads;
  float out[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int b = (tid >> 4) + 16 * e;
    out[e] = 0.f;
    if (b >= T) continue;
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = part[0][r][b][n];
#pragma unroll
      for (int w = 1; w < kFewWarps; ++w) s[r] += part[w][r][b][n];
    }
    out[e] = GATED ? f8_swiglu(s[0], s[R - 1]) : s[0];
    const int row = b;
    if (row >= p.M || n0 + n >= p.N) continue;
    if (p.y) p.y[row * p.y_stride + n0 + n] = f2bf(out[e]);
    if (p.yf) p.yf[row * p.y_stride + n0 + n] = out[e];
  }
  if (!GATED || !p.h) return;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int b = (tid >> 4) + 16 * e;
    uint32_t m = n0 + n < p.N ? __float_as_uint(out[e]) & 0x7fffffffu : 0u;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
    if (n == 0 && b < T) most[b] = m;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  uint32_t top[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int b = (tid >> 4) + 16 * e;
    uint32_t m = 0;
    if (b < T && n < kFewCluster) {  // lanes 0..7 of a row ask one CTA each
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc_smem(&most[b])), "r"(n));
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(m) : "r"(at) : "memory");
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
    top[e] = m;
  }
  // peers have read this CTA's maxima before it ends
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int b = (tid >> 4) + 16 * e, row = b;
    const bool fine = f8_finite(top[e]);
    const int byte = fine ? f8_scale_byte(top[e]) : kF8One;
    const uint32_t code = fine ? f8_codes4(out[e] * f8_inverse(byte), 0.f, 0.f, 0.f) & 0xffu : kF8Nan4 & 0xffu;
    if (b >= T || row >= p.M || n0 + n >= p.N) continue;
    p.h[row * p.h_stride + n0 + n] = (uint8_t)code;
    if (n == 0 && n0 % kF8Block == 0) p.hs[row * p.hs_stride + n0 / kF8Block] = (uint8_t)byte;
  }
}

template <int NT, bool GATED>
static cudaError_t few(const F8Prod& p, cudaStream_t s) {
  const int tiles = (p.N + 15) / 16;
  const bool cluster = GATED && p.h;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster ? (tiles + kFewCluster - 1) / kFewCluster * kFewCluster : tiles);
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kFewCluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_f8_few<NT, GATED>, p);
}

// At most 32 rows of x.
cudaError_t launch_f8_few(const F8Prod& p, bool gated, cudaStream_t s) {
  if (p.M <= 8) return gated ? few<1, true>(p, s) : few<1, false>(p, s);
  if (p.M <= 16) return gated ? few<2, true>(p, s) : few<2, false>(p, s);
  if (p.M <= 32) return gated ? few<4, true>(p, s) : few<4, false>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace bgq
