// gdn_device.h -- what is set up once on each device (kernel attributes hold for one device).
#pragma once

#include <atomic>

namespace gdn {

// run(device, set) calls set(), which returns 0 when it has succeeded, until it has done so on this
// device: a failure is reported and not kept.  Concurrent first calls may both set.
class OncePerDevice {
 public:
  template <typename F>
  int run(int device, F set) {
    const bool known = device >= 0 && device < kMax;
    if (known && done_[device].load(std::memory_order_acquire)) return 0;
    const int rc = set();
    if (rc == 0 && known) done_[device].store(true, std::memory_order_release);
    return rc;
  }

 private:
  static constexpr int kMax = 64;     // beyond them it is set on every call
  std::atomic<bool> done_[kMax] = {};
};

}  // namespace gdn
