// la2_bulk.cuh -- bulk copies between global and shared memory (16-byte
// granules, no data through registers) and the bounded wait for them.
#pragma once

#include "la2_common.cuh"
#include "la2_sm100.cuh"

namespace la2 {
namespace bulk {

using namespace sm100;

// Global to shared memory, counted by the mbarrier `bar`.
__device__ __forceinline__ void load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
// Shared to global memory, in the thread's current group of stores.
__device__ __forceinline__ void store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}
// Waits until all but this thread's newest group of bulk stores have read
// their source.
__device__ __forceinline__ void wait_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

// Bounded wait for phase `parity` of an mbarrier, as sm100::mbar_wait, but
// timed by the SM's clock: these kernels wait once for every row or slab, and
// reading the global timer each time costs more than most of the waits.
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      raise_error(ERR_TIMEOUT);
      return false;
    }
  }
}

}  // namespace bulk
}  // namespace la2
