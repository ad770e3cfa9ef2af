// kvp_wait.cuh -- mbarriers of the paged cache's attention, and waits on them
// that end by themselves.
#pragma once

#include <stdint.h>

namespace sf {

constexpr unsigned long long kWaitNs = 1000000000ull;  // waits give up after 1 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase for at most kWaitNs and counts itself in *timeouts where that
// runs out; after one wait of the CTA has given up none waits any more, and the CTA
// runs to its end without a result.
__device__ __forceinline__ void mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                               unsigned int* timeouts) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try(bar, parity)) {
    if (*gave_up) return;
    if (now_ns() - t0 > kWaitNs) {
      *gave_up = 1;
      atomicAdd(timeouts, 1u);
      return;
    }
  }
}
__device__ __forceinline__ void mbar_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up, unsigned int* timeouts) {
  if (!mbar_try(bar, parity)) mbar_wait_slow(bar, parity, gave_up, timeouts);
}
// A warp's wait for the work that it has in flight itself, before what that work
// uses is given back: not cut short by another wait that has given up.  One that
// runs out is counted once.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity, unsigned int* timeouts) {
  bool done = mbar_try(bar, parity);
  for (const unsigned long long t0 = now_ns(); !done && now_ns() - t0 <= kWaitNs;) done = mbar_try(bar, parity);
  if (!__all_sync(0xffffffffu, done) && (threadIdx.x & 31) == 0) atomicAdd(timeouts, 1u);
}

}  // namespace sf
