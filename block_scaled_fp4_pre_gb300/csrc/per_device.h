// State that a launcher finds out once and keeps: a kernel's raised shared-memory limit, the
// blocks that fit.  Both belong to a device, so there is one of each for every device that a
// process uses.  (No CUDA here: a device is its number.)
#pragma once

#include <atomic>

namespace mxmoe {

template <typename T>
class PerDevice {
 public:
  static constexpr int kMost = 64;
  // What is known of device `dev`, T() if nothing; nothing is kept of devices past kMost.
  T get(int dev) const {
    return dev >= 0 && dev < kMost ? v_[dev].load(std::memory_order_relaxed) : T();
  }
  void set(int dev, T v) {
    if (dev >= 0 && dev < kMost) v_[dev].store(v, std::memory_order_relaxed);
  }

 private:
  std::atomic<T> v_[kMost] = {};
};

// f(), which returns 0 on success, unless it has succeeded on this device; its result.
template <typename F>
auto once_a_device(PerDevice<bool>& done, int dev, F f) -> decltype(f()) {
  if (done.get(dev)) return {};
  const auto e = f();
  if (e == decltype(f())()) done.set(dev, true);
  return e;
}

}  // namespace mxmoe
