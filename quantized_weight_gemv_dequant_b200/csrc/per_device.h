// per_device.h -- numbers that belong to a device and are asked for once (host code only).
#pragma once

#include <atomic>

namespace ntx {

template <int N>
class PerDevice {
 public:
  // Number i of device `dev`, as ask(&value) gives it: 0 for success, anything else is returned and
  // asked for again.  Devices past the 64th are asked every time.
  template <class Ask>
  auto get(int dev, int i, int* value, Ask ask) -> decltype(ask(value)) {
    using Rc = decltype(ask(value));
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && (*value = kept_[dev][i].load(std::memory_order_relaxed)) != 0) {
      --*value;
      return Rc(0);
    }
    const Rc rc = ask(value);
    if (rc == Rc(0) && kept) kept_[dev][i].store(*value + 1, std::memory_order_relaxed);
    return rc;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> kept_[kDevices][N] = {};  // 1 more than the number; 0: not asked yet
};

}  // namespace ntx
