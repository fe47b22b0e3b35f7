// la2_memo.h -- answers about a device, kept for the next call.  Plain C++.
#pragma once

#include <stdint.h>

#include <atomic>

namespace la2 {

// The last answer (1 to 255) of each of the first 64 devices with the key that
// it was asked for: host threads and devices may take turns.  Another key or
// device asks again; so does a question that failed, whose stand-in is not kept.
class DeviceMemo {
  static constexpr int kDevices = 64;
  std::atomic<uint64_t> last_[kDevices] = {};  // key << 8 | answer; 0: none

 public:
  // ask(&n): whether there is an answer, and it
  template <typename Ask>
  int get(int device, uint64_t key, int stand_in, Ask &&ask) {
    const bool kept = device >= 0 && device < kDevices;
    if (kept) {
      const uint64_t known = last_[device].load(std::memory_order_relaxed);
      if (known && known >> 8 == key) return (int)(known & 255);
    }
    int n = 0;
    if (!ask(&n) || n < 1) return stand_in;
    if (n > 255) n = 255;
    if (kept) last_[device].store(key << 8 | (uint64_t)n, std::memory_order_relaxed);
    return n;
  }
};

}  // namespace la2
