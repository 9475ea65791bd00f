// f8_quant.cu — values into e4m3 codes with a power of two for each block: the
// quantiser, and the norm between a layer's halves (residual's addition, RMSNorm,
// quantisation in one pass over the row).
//
// Both are bound by memory: 3 bytes a value (2 read, 1 written), and 11 (h read and
// written, a bf16 addend read, a code written; 2 more for the bf16 copy).
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
// A CTA takes a row, a warp whole blocks of 128 columns of it (a lane 4 columns: loads and stores of a warp lie
// side by side, and a block's largest magnitude is one warp-wide maximum). With V blocks a warp the row stays in registers
// between the sum of squares and its use; with V = 0 (rows of more than 32 * 4 blocks) each thread reads back what it wrote.
template <int V, bool F32>
__global__ void __launch_bounds__(1024)
    k_rmsnorm_f8(float* h, const void* delta, const uint16_t* rho, int d, float eps, uint8_t* q, int64_t q_stride,
                 uint8_t* scale, int64_t s_stride, uint16_t* a) {
  __shared__ float part[32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, blocks = (d + kF8Block - 1) / kF8Block;
  const size_t row = blockIdx.x;
  float* hr = h + row * d;
  auto load = [&](int col) {
    float4 v = *reinterpret_cast<const float4*>(hr + col);
    if (delta) {
      float4 w;
      if (F32) {
        w = *reinterpret_cast<const float4*>(static_cast<const float*>(delta) + row * d + col);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(delta) + row * d + col);
        w = make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
      }
      v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    }
    return v;
  };
  auto squares = [](float4 v, float s) { return fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, s)))); };
  float4 v[V ? V : 1];
  float ss = 0.f;
  if (V) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (warp + i * warps) * kF8Block + lane * 4;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (col < d) v[i] = load(col);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (warp + i * warps) * kF8Block + lane * 4;
      ss = squares(v[i], ss);
      if (delta && col < d) *reinterpret_cast<float4*>(hr + col) = v[i];
    }
  } else {
    for (int b = warp; b < blocks; b += warps) {
      const int col = b * kF8Block + lane * 4;
      if (col >= d) break;
      const float4 w = load(col);
      ss = squares(w, ss);
      if (delta) *reinterpret_cast<float4*>(hr + col) = w;
    }
  }
  ss = warp_sum(ss);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  float sum = 0.f;
  for (int i = 0; i < warps; ++i) sum += part[i];
  const float r = 1.f / sqrtf(sum / (float)d + eps);
  auto finish = [&](int b, float4 w) {
    const int col = b * kF8Block + lane * 4;
    w = make_float4(w.x * r, w.y * r, w.z * r, w.w * r);
    if (rho && col < d) {
      const uint2 u = *reinterpret_cast<const uint2*>(rho + col);
      w = make_float4(w.x * bf16lo(u.x), w.y * bf16hi(u.x), w.z * bf16lo(u.y), w.w * bf16hi(u.y));
    }
    const uint32_t most = 0x7fffffffu;
    const uint32_t m = max(max(__float_as_uint(w.x) & most, __float_as_uint(w.y) & most),
                           max(__float_as_uint(w.z) & most, __float_as_uint(w.w) & most));
    const uint32_t top = __reduce_max_sync(kFull, col < d ? m : 0u);
    if (col >= d) return;
    const bool fine = f8_finite(top);
    const int byte = fine ? f8_scale_byte(top) : kF8One;
    const float inv = f8_inverse(byte);
    *reinterpret_cast<uint32_t*>(q + row * q_stride + col) =
        fine ? f8_codes4(w.x * inv, w.y * inv, w.z * inv, w.w * inv) : kF8Nan4;
    if (lane == 0) scale[row * s_stride + b] = (uint8_t)byte;
    if (a)
      *reinterpret_cast<uint2*>(a + row * d + col) = make_uint2((uint32_t)f2bf(w.x) | ((uint32_t)f2bf(w.y) << 16),
                                                                (uint32_t)f2bf(w.z) | ((uint32_t)f2bf(w.w) << 16));
  };
  if (V) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (warp + i * warps < blocks) finish(warp + i * warps, v[i]);
  } else {
    for (int b = warp; b < blocks; b += warps) {
      const int col = b * kF8Block + lane * 4;
      finish(b, col < d ? *reinterpret_cast<const float4*>(hr + col) : make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
}

template <bool F32>
static cudaError_t norm_by_size(float* h, const void* delta, const uint16_t* rho, float eps, const bgq_f8matrix& m,
                                uint16_t* a, cudaStream_t s) {
  const int blocks = f8_blocks(m.cols);
  auto go = [&](auto kern, int warps) {
    return launch_overlapped(kern, m.rows, warps * 32, 0, s, h, delta, rho, m.cols, eps, m.q, m.q_stride, m.scale,
                             m.scale_stride, a);
  };
  if (blocks <= 8) return go(k_rmsnorm_f8<1, F32>, blocks);
  if (blocks <= 16) return go(k_rmsnorm_f8<2, F32>, (blocks + 1) / 2);
  if (blocks <= 128) return go(k_rmsnorm_f8<4, F32>, (blocks + 3) / 4);
  return go(k_rmsnorm_f8<0, F32>, 32);
}

cudaError_t launch_rmsnorm_f8(float* h, const void* delta, bool delta_f32, const uint16_t* rho, float eps,
                              const bgq_f8matrix& m, uint16_t* a, cudaStream_t s) {
  return delta_f32 ? norm_by_size<true>(h, delta, rho, eps, m, a, s) : norm_by_size<false>(h, delta, rho, eps, m, a, s);
}

}  // namespace bgq
