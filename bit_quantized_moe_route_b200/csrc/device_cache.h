// A positive number that is found out once for each device (host code).
#pragma once

#include <atomic>

namespace moe {

class DeviceCache {
 public:
  // query() gives the number, or 0 or less if it has none: that is not kept, so
  // a failure that passes is asked again by the next call.
  template <typename F>
  int get(int device, F&& query) {
    const bool kept = device >= 0 && device < kDevices;
    int v = kept ? v_[device].load(std::memory_order_acquire) : 0;
    if (v < 1) {
      v = query();
      if (kept && v > 0) v_[device].store(v, std::memory_order_release);
    }
    return v;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> v_[kDevices] = {};
};

}  // namespace moe
