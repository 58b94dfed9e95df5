// A number per device that is found out once (host only).
#pragma once

#include <atomic>

namespace moe {

// Any number of host threads may ask at once: those that come before the first
// answer each find it out, and no thread sees a half-written one.
class DeviceCache {
 public:
  // The number of device `dev`: find() >= 0 at the first call; 0 while find()
  // fails (< 0, not kept) and for devices past the table.
  template <typename F>
  int get(int dev, F&& find) {
    if (dev < 0 || dev >= kDevices) return 0;
    int v = known_[dev].load(std::memory_order_acquire);
    if (v == 0) {
      const int n = find();
      if (n < 0) return 0;
      v = n + 1;
      known_[dev].store(v, std::memory_order_release);
    }
    return v - 1;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices] = {};  // the number + 1; 0: not known
};

}  // namespace moe
