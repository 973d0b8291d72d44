// A property of a kernel or GPU that is looked up once per device, from any
// thread. Host only, plain C++.
#pragma once

#include <atomic>

namespace dsmoe {

class PerDevice {
 public:
  // The value of device `dev`, or find() where it is not known yet (several
  // threads may then find it; they find the same). find() > 0.
  template <class Find>
  int get(int dev, Find&& find) {
    if (dev < 0 || dev >= kDevices) return find();
    int v = value_[dev].load(std::memory_order_relaxed);
    if (!v) {
      v = find();
      value_[dev].store(v, std::memory_order_relaxed);
    }
    return v;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> value_[kDevices] = {};
};

}  // namespace dsmoe
