// A number that each device answers once (host code only).
#pragma once

#include <atomic>

namespace moe {

class PerDevice {
 public:
  // What `query` answered for this device: it is asked until it does, a
  // negative answer is a failure (0 to the caller) and is not kept.
  template <class Query>
  int get(int device, Query query) {
    if (device < 0 || device >= kDevices) return 0;
    int n = known_[device].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    n = query();
    if (n < 0) return 0;
    known_[device].store(n + 1, std::memory_order_relaxed);  // (0: not known)
    return n;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices] = {};
};

}  // namespace moe
