// What holds for one device and is looked up or set once on each: kernels' shared-memory
// limits, counts of SMs and clusters. (A function's static would hold what the device
// said, or failed to, that called first.) Any thread may call; what two find at a time is
// the same. Plain C++, so that it is tested on a host without a device.
#pragma once

#include <stdint.h>

#include <atomic>

namespace gdn {

constexpr int kMaxDevices = 64;          // others look it up at every call

// Runs what has not succeeded yet on the device: a status that equals Status{} (cudaSuccess)
// is kept, a failure is not.
class DeviceOnce {
 public:
  template <typename F>
  auto operator()(int device, F set) -> decltype(set()) {
    using Status = decltype(set());
    const uint64_t bit = device >= 0 && device < kMaxDevices ? 1ull << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return Status{};
    const Status s = set();
    if (s == Status{}) done_.fetch_or(bit, std::memory_order_release);
    return s;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// A number above 0 that each device has; what is not is not kept.
class DeviceNumber {
 public:
  template <typename F>
  int operator()(int device, F find) {
    const bool known = device >= 0 && device < kMaxDevices;
    int n = known ? n_[device].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    n = find();
    if (known && n > 0) n_[device].store(n, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<int> n_[kMaxDevices] = {};
};

}  // namespace gdn
