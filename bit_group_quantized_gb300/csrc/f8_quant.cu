// f8_quant.cu — values into e4m3 codes with a power of two for each block: the
// quantiser, and the norm between a layer's halves (residual's addition, RMSNorm,
// quantisation in one pass over the row).
//
// Both are bound by memory: 3 bytes a value (2 read, 1 written), and 11 (h read and
// written, a bf16 addend read, a code written; 2 more for the bf16 copy). Measured (a graph of calls over more than L2
// holds): quantiser 12288 x 4096 in blocks 22.7 us, 6.6 TB/s; 4097 x 8192 in rows 17.0 us, 5.9 TB/s; norm 8191 x 4096 56.0 us, 6.6
// TB/s; 2049 x 5008 with fp32 addend and bf16 copy 28.1 us, 5.5 TB/s, where 2.2 waves of CTAs take the time of three.
#include <type_traits>

#include "common.cuh"
#include "f8.h"
#include "kernels.h"

namespace bgq {

// ------------------------------------------------------------------ quantiser
// Scales for 128 columns of a row: a lane has 8 columns (one 16-byte load), 16 lanes a
// block, a warp 256 columns of a row, and kQuantUnits such pieces, all loaded first. Largest magnitudes are
// found on the bf16 bits, two at a time; NaN and infinities are then the largest.
constexpr int kQuantWarps = 8, kQuantUnits = 4;

__device__ __forceinline__ uint32_t f8_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// The codes of 8 bf16 values; `inv` as f8_inverse's.
__device__ __forceinline__ uint2 f8_codes8(uint4 v, float inv) {
  return make_uint2(f8_codes4(bf16lo(v.x) * inv, bf16hi(v.x) * inv, bf16lo(v.y) * inv, bf16hi(v.y) * inv),
                    f8_codes4(bf16lo(v.z) * inv, bf16hi(v.z) * inv, bf16lo(v.w) * inv, bf16hi(v.w) * inv));
}

__global__ void __launch_bounds__(kQuantWarps * 32)
    k_f8_quantise(const uint16_t* x, int64_t x_stride, uint8_t* q, int64_t q_stride, uint8_t* scale, int64_t s_stride,
                  int cols, uint32_t pieces, uint32_t units) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint64_t first = ((uint64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5)) * kQuantUnits;
  if (first >= units) return;
  uint32_t row[kQuantUnits];
  int col[kQuantUnits];
  row[0] = (uint32_t)first / pieces;
  uint32_t piece = (uint32_t)first - row[0] * pieces;
  uint4 v[kQuantUnits];
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    col[i] = first + i < units ? (int)piece * 256 + lane * 8 : cols;
    v[i] = make_uint4(0, 0, 0, 0);
    if (col[i] < cols) v[i] = *reinterpret_cast<const uint4*>(x + row[i] * x_stride + col[i]);
    if (i + 1 < kQuantUnits) {
      const bool next = ++piece == pieces;
      row[i + 1] = row[i] + next;
      if (next) piece = 0;
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    uint32_t m = f8_max2(f8_max2(f8_max2(v[i].x & 0x7fff7fffu, v[i].y), v[i].z), v[i].w);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kFull, m, o));
    const uint32_t top = max(m & 0xffffu, m >> 16) << 16;
    if (col[i] >= cols) continue;
    const bool fine = f8_finite(top);
    const int byte = fine ? f8_scale_byte(top) : kF8One;
    uint2 c = make_uint2(kF8Nan4, kF8Nan4);
    if (fine) c = f8_codes8(v[i], f8_inverse(byte));
    *reinterpret_cast<uint2*>(q + row[i] * q_stride + col[i]) = c;
    if ((lane & 15) == 0) scale[row[i] * s_stride + (col[i] >> 7)] = (uint8_t)byte;
  }
}

// Scales for 128 x 128 values: a CTA has one block in registers, a thread 16 columns of 4 rows.
__global__ void __launch_bounds__(256)
    k_f8_quantise_block(const uint16_t* x, int64_t x_stride, uint8_t* q, int64_t q_stride, uint8_t* scale,
                        int64_t s_stride, int rows, int cols, int across) {
  __shared__ uint32_t most[8];
  pdl_wait();
  pdl_trigger();
  const int down = blockIdx.x / across, b = blockIdx.x - down * across;
  const int col = b * kF8Block + (threadIdx.x & 7) * 16, row = down * kF8Block + (threadIdx.x >> 3);
  uint4 v[4][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v[i][j] = make_uint4(0, 0, 0, 0);
      if (row + 32 * i < rows && col < cols)
        v[i][j] = *reinterpret_cast<const uint4*>(x + (row + 32 * i) * x_stride + col + 8 * j);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) m = f8_max2(f8_max2(f8_max2(f8_max2(m, v[i][j].x), v[i][j].y), v[i][j].z), v[i][j].w);
  m = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, most[i]);
  const uint32_t top = m << 16;
  const bool fine = f8_finite(top);
  const int byte = fine ? f8_scale_byte(top) : kF8One;
  if (threadIdx.x == 0) scale[down * s_stride + b] = (uint8_t)byte;
  const float inv = f8_inverse(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row + 32 * i >= rows || col >= cols) continue;
    uint4 c = make_uint4(kF8Nan4, kF8Nan4, kF8Nan4, kF8Nan4);
    if (fine) {
      const uint2 lo = f8_codes8(v[i][0], inv), hi = f8_codes8(v[i][1], inv);
      c = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    *reinterpret_cast<uint4*>(q + (row + 32 * i) * q_stride + col) = c;
  }
}

cudaError_t launch_f8_quantise(const uint16_t* x, int64_t x_stride, const bgq_f8matrix& m, cudaStream_t s) {
  if (m.block_rows == 1) {
    const uint32_t pieces = (m.cols + 255) / 256, units = pieces * (uint32_t)m.rows;  // below 2^8 and 2^32
    const int per = kQuantWarps * kQuantUnits;
    return launch_overlapped(k_f8_quantise, (int)(((uint64_t)units + per - 1) / per), kQuantWarps * 32, 0, s, x, x_stride,
                             m.q, m.q_stride, m.scale, m.scale_stride, m.cols, pieces, units);
  }
  const int across = f8_blocks(m.cols), down = f8_blocks(m.rows);
  return launch_overlapped(k_f8_quantise_block, across * down, 256, 0, s, x, x_stride, m.q, m.q_stride, m.scale,
                           m.scale_stride, m.rows, m.cols, across);
}

// ----------------------------------------------------------------------- norm
// A warp has whole blocks of 128 columns of a row (a lane 4 columns: loads and stores of a warp lie side by side, and a block's
// largest magnitude is one warp-wide maximum), V of them, which stay in registers between the sum of squares and its use. A
// row is a warp's alone (ALONE: up to 8 blocks) or a CTA's. (CTAs that walk through the rows and load the next one meanwhile
// need twice the registers: 8191 x 4096 took 75 us, 60 so.)
template <bool F32>
struct NormRaw {
  float4 h;
  typename std::conditional<F32, float4, uint2>::type delta;
};

struct NormArgs {
  float* h;
  const void* delta;
  const uint16_t* rho;
  uint8_t* q;
  uint8_t* scale;
  uint16_t* a;
  int64_t q_stride, s_stride;
  int rows, d;
  float eps;
};

__device__ __forceinline__ float norm_squares(float4 v, float s) {
  return fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, s))));
}
template <bool F32>
__device__ __forceinline__ float4 norm_sum(const NormArgs& n, const NormRaw<F32>& r) {
  float4 v = r.h;
  if (n.delta) {
    if constexpr (F32)
      v = make_float4(v.x + r.delta.x, v.y + r.delta.y, v.z + r.delta.z, v.w + r.delta.w);
    else
      v = make_float4(v.x + bf16lo(r.delta.x), v.y + bf16hi(r.delta.x), v.z + bf16lo(r.delta.y), v.w + bf16hi(r.delta.y));
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ void norm_load(const NormArgs& n, int64_t row, int col, NormRaw<F32>& r) {
  r.h = *reinterpret_cast<const float4*>(n.h + row * n.d + col);
  if (n.delta) {
    if constexpr (F32)
      r.delta = *reinterpret_cast<const float4*>(static_cast<const float*>(n.delta) + row * n.d + col);
    else
      r.delta = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(n.delta) + row * n.d + col);
  }
}
// One block of a row by one warp: w times r and rho, as codes and, where wanted, in bf16.
__device__ __forceinline__ void norm_finish(const NormArgs& n, int64_t row, int b, float4 w, float r, uint2 rho) {
  const int lane = threadIdx.x & 31, col = b * kF8Block + lane * 4;
  w = make_float4(w.x * r, w.y * r, w.z * r, w.w * r);
  if (n.rho) w = make_float4(w.x * bf16lo(rho.x), w.y * bf16hi(rho.x), w.z * bf16lo(rho.y), w.w * bf16hi(rho.y));
  const uint32_t most = 0x7fffffffu;
  const uint32_t m = max(max(__float_as_uint(w.x) & most, __float_as_uint(w.y) & most),
                         max(__float_as_uint(w.z) & most, __float_as_uint(w.w) & most));
  const uint32_t top = __reduce_max_sync(kFull, col < n.d ? m : 0u);
  if (col >= n.d) return;
  const bool fine = f8_finite(top);
  const int byte = fine ? f8_scale_byte(top) : kF8One;
  const float inv = f8_inverse(byte);
  *reinterpret_cast<uint32_t*>(n.q + row * n.q_stride + col) = fine ? f8_codes4(w.x * inv, w.y * inv, w.z * inv, w.w * inv) : kF8Nan4;
  if (lane == 0) n.scale[row * n.s_stride + b] = (uint8_t)byte;
  if (n.a)
    *reinterpret_cast<uint2*>(n.a + row * n.d + col) = make_uint2((uint32_t)f2bf(w.x) | ((uint32_t)f2bf(w.y) << 16),
                                                                  (uint32_t)f2bf(w.z) | ((uint32_t)f2bf(w.w) << 16));
}

template <int V, bool F32, bool ALONE>
__global__ void __launch_bounds__(ALONE ? 256 : 512, V == 8 && !ALONE ? 2 : 1) k_rmsnorm_f8(const NormArgs n) {
  __shared__ float part[32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, blocks = (n.d + kF8Block - 1) / kF8Block;
  // the row's blocks that this warp has: first, first + step, ...
  const int first = ALONE ? 0 : warp, step = ALONE ? 1 : warps;
  const int64_t row = ALONE ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
  if (ALONE && row >= n.rows) return;
  float4 v[V];
  float ss = 0.f;
  {
    NormRaw<F32> raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (first + i * step) * kF8Block + lane * 4;
      raw[i] = {};
      if (col < n.d) norm_load<F32>(n, row, col, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (first + i * step) * kF8Block + lane * 4;
      v[i] = norm_sum<F32>(n, raw[i]);  // zeros past the row's end
      ss = norm_squares(v[i], ss);
      if (n.delta && col < n.d) *reinterpret_cast<float4*>(n.h + row * n.d + col) = v[i];
    }
  }
  ss = warp_sum(ss);
  if (!ALONE) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < warps; ++i) ss += part[i];
  }
  const float r = 1.f / sqrtf(ss / (float)n.d + n.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int b = first + i * step, col = b * kF8Block + lane * 4;
    if (b < blocks) norm_finish(n, row, b, v[i], r, n.rho && col < n.d ? *reinterpret_cast<const uint2*>(n.rho + col) : make_uint2(0, 0));
  }
}

// Rows of more than 128 blocks: each thread reads back what it wrote.
template <bool F32>
__global__ void __launch_bounds__(1024) k_rmsnorm_f8_long(const NormArgs n) {
  __shared__ float part[32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, blocks = (n.d + kF8Block - 1) / kF8Block;
  const int64_t row = blockIdx.x;
  float ss = 0.f;
#pragma unroll 4
  for (int b = warp; b < blocks; b += warps) {
    const int col = b * kF8Block + lane * 4;
    if (col >= n.d) break;
    NormRaw<F32> raw;
    norm_load<F32>(n, row, col, raw);
    const float4 v = norm_sum<F32>(n, raw);
    ss = norm_squares(v, ss);
    if (n.delta) *reinterpret_cast<float4*>(n.h + row * n.d + col) = v;
  }
  ss = warp_sum(ss);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = 0.f;
  for (int i = 0; i < warps; ++i) ss += part[i];
  const float r = 1.f / sqrtf(ss / (float)n.d + n.eps);
  for (int b = warp; b < blocks; b += warps) {
    const int col = b * kF8Block + lane * 4;
    const bool there = col < n.d;
    norm_finish(n, row, b, there ? *reinterpret_cast<const float4*>(n.h + row * n.d + col) : make_float4(0.f, 0.f, 0.f, 0.f), r,
                there && n.rho ? *reinterpret_cast<const uint2*>(n.rho + col) : make_uint2(0, 0));
  }
}

template <bool F32>
static cudaError_t norm_by_size(const NormArgs& n, cudaStream_t s) {
  const int blocks = f8_blocks(n.d);
  auto alone = [&](auto kern) { return launch_overlapped(kern, (n.rows + 7) / 8, 256, 0, s, n); };
  auto rows = [&](auto kern, int warps) { return launch_overlapped(kern, n.rows, warps * 32, 0, s, n); };
  if (blocks <= 1) return alone(k_rmsnorm_f8<1, F32, true>);
  if (blocks <= 2) return alone(k_rmsnorm_f8<2, F32, true>);
  if (blocks <= 4) return alone(k_rmsnorm_f8<4, F32, true>);
  if (blocks <= 8) return alone(k_rmsnorm_f8<8, F32, true>);
  // few rows: more warps each (512 x 4096: 5.4 us so, 6.5 with four blocks a warp; 8191 x 4096: 58 and 56)
  if (blocks <= 32 && n.rows <= 4 * num_sms()) return rows(k_rmsnorm_f8<2, F32, false>, (blocks + 1) / 2);
  if (blocks <= 64) return rows(k_rmsnorm_f8<4, F32, false>, (blocks + 3) / 4);
  if (blocks <= 128) return rows(k_rmsnorm_f8<8, F32, false>, (blocks + 7) / 8);
  return launch_overlapped(k_rmsnorm_f8_long<F32>, n.rows, 1024, 0, s, n);
}

cudaError_t launch_rmsnorm_f8(float* h, const void* delta, bool delta_f32, const uint16_t* rho, float eps,
                              const bgq_f8matrix& m, uint16_t* a, cudaStream_t s) {
  const NormArgs n = {h, delta, rho, m.q, m.scale, a, m.q_stride, m.scale_stride, m.rows, m.cols, eps};
  return delta_f32 ? norm_by_size<true>(n, s) : norm_by_size<false>(n, s);
}

}  // namespace bgq
