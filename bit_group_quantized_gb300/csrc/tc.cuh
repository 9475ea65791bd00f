// tc.cuh — mbarriers, fences and tensor memory for the tcgen05 kernels
// (umma.cu, kv4_prompt.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace bgq {

__device__ __forceinline__ uint32_t tc_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ unsigned long long tc_time() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void tc_mbar_init(uint64_t* m, int count = 1) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(m)), "r"(count) : "memory");
}
__device__ __forceinline__ void tc_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc_smem(m)) : "memory");
}
__device__ __forceinline__ bool tc_mbar_try(uint64_t* m, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc_smem(m)), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same test, suspending the thread until the phase completes or
// kTcSuspendNs pass: waiting warps then leave the issue slots to the warps
// doing the work.
constexpr uint32_t kTcSuspendNs = 20000;
__device__ __forceinline__ bool tc_mbar_try_suspend(uint64_t* m, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc_smem(m)), "r"(parity), "r"(kTcSuspendNs)
      : "memory");
  return ok != 0;
}
// Bounded wait; false on timeout (the polling loop kept out of line).
static __device__ __noinline__ bool tc_mbar_wait_loop(uint64_t* m, uint32_t parity, long long limit_ns) {
  const unsigned long long t0 = tc_time();
  long long it = 0;
  while (!tc_mbar_try_suspend(m, parity)) {
    if ((long long)(tc_time() - t0) > limit_ns || ++it > (1ll << 28)) return false;
  }
  return true;
}
__device__ __forceinline__ bool tc_mbar_wait(uint64_t* m, uint32_t parity, long long limit_ns) {
  return tc_mbar_try(m, parity) || tc_mbar_wait_loop(m, parity, limit_ns);
}
__device__ __forceinline__ void tc_fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Tensor memory: allocation and release by one whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* m) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc_smem(m))
               : "memory");
}
}  // namespace bgq
