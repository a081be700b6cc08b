// What is set up once per device before a kernel's first launch there: its shared-memory
// attribute, the grid that can be resident.
#pragma once

#include <atomic>

namespace moe {

class PerDevice {
 public:
  // The device's value: what make(&value) gave at its first use there (not 0). Returns
  // make's error, the type's zero value meaning none; after an error the next call makes it
  // again. Host threads may call at once: each may make the value, all make the same.
  template <class Make>
  auto get(int device, int* value, Make make) -> decltype(make(value)) {
    using Error = decltype(make(value));
    const bool kept = device >= 0 && device < kDevices;
    if (kept) {
      *value = values_[device].load(std::memory_order_acquire);
      if (*value != 0) return Error{};
    }
    const Error e = make(value);
    if (e == Error{} && kept) values_[device].store(*value, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> values_[kDevices] = {};
};

}  // namespace moe
