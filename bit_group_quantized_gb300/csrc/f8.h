// f8.h — the e4m3 operators: arguments of their kernels, and device helpers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/bgq.h"
#include "f8_rule.h"

namespace bgq {

__host__ __device__ inline int f8_blocks(int cols) { return (cols + kF8Block - 1) / kF8Block; }

struct Ctrl;

// One product: y = x W^T, or silu(x W0^T) * (x W1^T) into h and / or y.
struct F8Prod {
  const uint8_t* w[2];   // codes of W, or of gate and up
  const uint8_t* ws[2];  // their scales
  int64_t w_stride[2], ws_stride[2];
  const uint8_t* x;
  const uint8_t* xs;
  int64_t x_stride, xs_stride;
  int M, N, K;  // rows of x, rows of W, columns of both
  uint16_t* y;
  float* yf;
  int64_t y_stride;
  uint8_t* h;  // codes of the result (gated), null where it is wanted in bf16 alone
  uint8_t* hs;
  int64_t h_stride, hs_stride;
  Ctrl* ctrl;
};

cudaError_t launch_f8_quantise(const uint16_t* x, int64_t x_stride, const bgq_f8matrix& m, cudaStream_t s);
cudaError_t launch_rmsnorm_f8(float* h, const void* delta, bool delta_f32, const uint16_t* rho, float eps,
                              const bgq_f8matrix& m, uint16_t* a, cudaStream_t s);
cudaError_t launch_f8_product(const F8Prod& p, bool gated, cudaStream_t s);
cudaError_t launch_f8_few(const F8Prod& p, bool gated, cudaStream_t s);
cudaError_t launch_f8_mid(const F8Prod& p, bool gated, const F8MidPlan& plan, cudaStream_t s);
cudaError_t launch_f8_many(const F8Prod& p, bool gated, cudaStream_t s);

#ifdef __CUDACC__
// The scale byte of a block whose largest magnitude has these fp32 bits: the smallest power of two 2^(byte - 127) with
// amax <= 448 * 2^(byte - 127). 448 = 1.75 * 2^8, so it goes by the exponent, one more where the fraction passes 1.75.
__device__ __forceinline__ int f8_scale_byte(uint32_t amax_bits) {
  return max(0, (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0));
}
__device__ __forceinline__ bool f8_finite(uint32_t amax_bits) { return amax_bits < 0x7f800000u; }
// 2^(127 - byte), by which the block's values are multiplied; bytes here are at most 247.
__device__ __forceinline__ float f8_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Four values as e4m3 codes, a in the lowest byte (to nearest, halves to even).
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
constexpr uint32_t kF8Nan4 = 0x7f7f7f7fu;  // four codes of NaN
constexpr int kF8One = 127;                // the scale byte of 1

// silu(g) * u for g >= kF8Far, or NaN. __expf is off by 2 + 1.2 |g| units of 2^-23 (at -64 some 2^-17), the reciprocal by one;
// the result has 8 bits or 4. At -64 the exponential is 2^92.
constexpr float kF8Far = -64.f;
__device__ __forceinline__ float f8_swiglu_near(float g, float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-g)));
  return g * r * u;
}
// Gates below kF8Far, where silu(g) is g exp(g) to fp32's last place, become kF8Far and u takes what that leaves out, g / -64
// exp(g + 64): exp(-g) itself leaves fp32 at -88.7, where a large u still makes an ordinary number of the product. The exponential comes in
// two halves, neither subnormal down to g = -238, where the result is below fp32's range whatever u is; it is less than one, and so is silu(-64), so
// nothing on the way is smaller than the result. Off by another 6 + |g + 64| units of 2^-23. Other gates stay as they are.
__device__ __forceinline__ void f8_nearer(float& g, float& u) {
  float t;  // exp((g + 64) / 2)
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"((g - kF8Far) * 0.72134752f));
  const bool far = g < kF8Far;
  u = far ? u * t * t * (g * (1.f / kF8Far)) : u;
  g = far ? kF8Far : g;
}
__device__ __forceinline__ float f8_swiglu(float g, float u) {
  if (g < kF8Far) f8_nearer(g, u);
  return f8_swiglu_near(g, u);
}
// Four of them with one branch, far gates being rare (a branch each: gated 64 x 2 * 1024 x 4096 took 6.9 us for 6.7).
__device__ __forceinline__ float4 f8_swiglu4(float4 g, float4 u) {
  if (fminf(fminf(g.x, g.y), fminf(g.z, g.w)) < kF8Far) {
    f8_nearer(g.x, u.x);
    f8_nearer(g.y, u.y);
    f8_nearer(g.z, u.z);
    f8_nearer(g.w, u.w);
  }
  return make_float4(f8_swiglu_near(g.x, u.x), f8_swiglu_near(g.y, u.y), f8_swiglu_near(g.z, u.z), f8_swiglu_near(g.w, u.w));
}
#endif

}  // namespace bgq
