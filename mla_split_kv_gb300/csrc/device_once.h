// What has to be set once for each device of a process (plain C++).
#pragma once

#include <atomic>
#include <cstdint>

namespace mla {

// Calls `set` on the current device `dev` until it has succeeded there once (returned its type's zero, cudaSuccess).
// Function attributes -- a kernel's shared-memory limit, clusters of more than 8 -- belong to a device, so a flag for
// the whole process would leave every device but the first without them. Threads that meet here may both set the same
// value. Devices past the mask's 64 are set every time.
class DeviceOnce {
 public:
  template <class Set>
  auto operator()(int dev, Set set) -> decltype(set()) {
    using Status = decltype(set());
    if (dev < 0 || dev > 63) return set();
    const uint64_t bit = uint64_t{1} << dev;
    if (done_.load(std::memory_order_relaxed) & bit) return Status{};
    const Status status = set();
    if (status == Status{}) done_.fetch_or(bit, std::memory_order_relaxed);
    return status;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace mla
