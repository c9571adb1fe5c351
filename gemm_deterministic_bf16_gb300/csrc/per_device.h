// per_device.h -- set-up that each device of the process needs once, such as a
// kernel's shared-memory limit: cudaFuncSetAttribute acts on the current device
// alone.
#pragma once

#include <stdint.h>

#include <atomic>

namespace detffn {

class PerDevice {
 public:
  static constexpr int kDevices = 64;   // (beyond these: set up at every call)

  // Calls set() unless it has succeeded (returned 0) for `device` before.  A
  // failure is returned and not kept: the next call tries again.  Host threads
  // that arrive together may both call it.
  template <class F>
  auto once(int device, F&& set) -> decltype(set()) {
    const bool kept = device >= 0 && device < kDevices;
    const uint64_t bit = kept ? 1ull << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return decltype(set())(0);
    const auto r = set();
    if (r == decltype(set())(0)) done_.fetch_or(bit, std::memory_order_release);
    return r;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace detffn
