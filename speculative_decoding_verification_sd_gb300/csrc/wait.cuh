// wait.cuh -- bounded waits on mbarrier phases.
#pragma once

#include "sd_device.cuh"

namespace sdk {

constexpr uint64_t kDrainNs = 2000000000ull;  // a drain of copies in flight gives up after this time

__device__ __forceinline__ uint64_t clock_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for a phase; false when `limit_ns` ran out first.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (phase_done(bar, parity)) return true;
  const uint64_t end = clock_ns() + limit_ns;
  while (!phase_done(bar, parity))
    if (clock_ns() > end) return false;
  return true;
}

}  // namespace sdk
