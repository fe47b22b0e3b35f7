// la2_bulk.cuh -- bulk copies between global and shared memory (16-byte
// granules, no data through registers).
#pragma once

#include <stdint.h>

namespace la2 {
namespace bulk {

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

}  // namespace bulk
}  // namespace la2
