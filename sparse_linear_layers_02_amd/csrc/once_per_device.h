// What has to be set on each device before its first use there, such as an
// attribute of a kernel, which belongs to the device that is current.
#pragma once

#include <atomic>
#include <cstdint>

namespace sbn {

class OncePerDevice {
 public:
  // set() returns 0 for success.  It runs on a device until it has succeeded
  // there, perhaps more than once if threads meet; its result, or 0 if it need not run.
  template <class Set>
  auto operator()(int device, Set set) -> decltype(set()) {
    const bool kept = device >= 0 && device < 64;
    const uint64_t bit = kept ? uint64_t(1) << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return {};
    const auto result = set();
    if (result == decltype(set()){}) done_.fetch_or(bit, std::memory_order_release);
    return result;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace sbn
