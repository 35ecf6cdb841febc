// What a device answered to a query, kept per device and key: devices of one compute capability may
// differ in what runs at once.
#pragma once

#include <atomic>

namespace moe {

constexpr int kCountDevices = 64;

template <int KEYS>
class DeviceCounts {
 public:
  // query() gives the count (0: the device does not do it), or a negative value where it
  // failed: that says nothing about the device, counts as 0 in this call and is asked again in the next.
  template <typename Query>
  int get(int device, int key, Query query) {
    if (device < 0 || device >= kCountDevices || key < 0 || key >= KEYS) return 0;
    std::atomic<int>& known = known_[device][key];
    int n = known.load(std::memory_order_relaxed) - 1;
    if (n < 0) {
      n = query();
      if (n < 0) return 0;
      known.store(n + 1, std::memory_order_relaxed);
    }
    return n;
  }

 private:
  std::atomic<int> known_[kCountDevices][KEYS] = {};  // the count and one more; 0: not asked yet
};

}  // namespace moe
