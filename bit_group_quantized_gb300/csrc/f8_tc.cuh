// f8_tc.cuh — what the tcgen05 kernels of e4m3 products share: operand tiles, scaled
// matrix instructions, bounded waits.
//
// Operand tiles are 128 rows of 128 bytes (one block of columns), brought by TMA in the 128-byte
// swizzled layout. The matrix instruction (kind::mxf8f6f4, 32 columns a step) takes a power-of-two scale for each row of both
// operands from tensor memory: row 32 j + l of 128 in lane l (of each 32 lanes, four times alike) and column
// j, four scales a word, of which the instruction names one. One scale stands for 32 columns there and for 128 here, so four
// steps name the same one, and a word serves four blocks: 512 columns.
#pragma once

#include <atomic>

#include "common.cuh"
#include "f8.h"
#include "kernels.h"
#include "tc.cuh"
#include "tc_map.h"

namespace bgq {

constexpr long long kF8TimeoutNs = 1000000000ll;
constexpr int kF8Tile = 128 * 128;  // bytes of an operand tile

// Bounded wait: on expiry, or once *fail is set elsewhere, it returns false and *fail is set.
static __device__ __noinline__ bool f8_wait_loop(uint64_t* m, uint32_t parity, volatile int* fail) {
  const unsigned long long t0 = tc_time();
  long long it = 0;
  while (!tc_mbar_try_suspend(m, parity)) {
    if (*fail) return false;
    if ((long long)(tc_time() - t0) > kF8TimeoutNs || ++it > (1ll << 28)) {
      *fail = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool f8_wait(uint64_t* m, uint32_t parity, volatile int* fail) {
  return tc_mbar_try(m, parity) || f8_wait_loop(m, parity, fail);
}
// The address of something of this CTA's shared memory in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t f8_at(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc_smem(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t f8_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// An arrival at a barrier of either CTA. What it tells of is tensor memory, which tcgen05's own fences order; released for the
// whole cluster it would wait for every load in flight (2000 cycles for each set of scales).
__device__ __forceinline__ void f8_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void f8_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void f8_expect(uint64_t* m, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(m)), "r"(bytes) : "memory");
}

// CG: CTAs that share a matrix instruction. With two, each brings its half of both operands to its own
// shared memory and tells the first one's barrier.
template <int CG>
__device__ __forceinline__ void f8_load(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            tc_smem(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            tc_smem(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void f8_map_ahead(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Tensor memory of both CTAs of a pair, by one whole warp of each (of a single CTA: tc.cuh).
__device__ __forceinline__ void f8_tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void f8_tmem_free(uint32_t at, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
// Issued by the lane that has `lead`; the whole warp runs the code around them, so that addresses and descriptors stay
// in uniform registers.
__device__ __forceinline__ uint32_t f8_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
template <int CG>
__device__ __forceinline__ void f8_commit(uint64_t* m, uint32_t lead) {  // with two CTAs: the barrier of both
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(tc_smem(m)),
        "h"((uint16_t)3), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc_smem(m)),
        "r"(lead)
        : "memory");
}

// K-major operand in the 128-byte swizzled layout: 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t f8_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// e4m3 x e4m3 -> fp32, e8m0 scales, number `sf` of their words, M x N.
__device__ __forceinline__ uint32_t f8_idesc(int m, int n, int sf) {
  return ((uint32_t)sf << 4) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24) | ((uint32_t)sf << 29);
}
template <int CG>
__device__ __forceinline__ void f8_tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t acc,
                                          uint32_t lead) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(lead)
        : "memory");
}

// 4 words of a thread's lane into columns from `at`; 32 fp32 columns of it.
__device__ __forceinline__ void f8_tmem_st4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void f8_tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void f8_tmem_ld32(uint32_t at, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void f8_tmem_ld16(uint32_t at, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void f8_tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Lets a kernel have `most` bytes of dynamic shared memory: asked for once a device (`known`: a bit for each).
inline cudaError_t f8_room(const void* kern, int most, std::atomic<uint64_t>& known) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && known.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess && dev < 64) known.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// The tensor map of codes [rows][cols], in tiles of `box_rows` rows and 128 columns; zeros beyond both ends.
inline bool f8_map(CUtensorMap* m, const uint8_t* q, int rows, int cols, int64_t stride, int box_rows = 128) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------ results
// A warp writes 32 rows of 128 bytes at a time, a row a thread, by way of shared memory and a TMA store, which also cuts them where
// the matrix ends: a thread's own 16-byte stores touch 32 lines at a time, and a tile's took 2 us.
// The room is 4096 bytes, 1024-byte aligned, in the 128-byte swizzled layout; a warp has two.
constexpr int kF8Room = 32 * 128;
__device__ __forceinline__ void f8_store_rows(unsigned char* room, const uint4 (&line)[8], const CUtensorMap* map, int col, int row) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the store before the last has read this room
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(room + lane * 128 + ((i ^ lane) & 7) * 16) = line[i];
  tc_fence_proxy();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(tc_smem(room))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void f8_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// The least of three (a NaN only if all are), and the largest magnitude of three (a NaN if one is).
__device__ __forceinline__ float f8_min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float f8_most3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint4 f8_bf16x8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = (uint32_t)f2bf(v[2 * j]) | ((uint32_t)f2bf(v[2 * j + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 f8_fp32x4(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
// The tensor map of a result of `size` bytes a value, in pieces of 32 rows of 128 bytes.
inline bool f8_out_map(CUtensorMap* m, void* y, int size, int rows, int cols, int64_t stride) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(stride * size)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32}, es[2] = {1, 1};
  const CUtensorMapDataType type = size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32;
  return enc(m, type, 2, y, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace bgq
