// What a launch asks the driver once for each device and keeps.  (Plain C++, so that it can be
// checked on the host.)
#pragma once

#include <atomic>

namespace flexq {

// A positive number that belongs to a device: a kernel's registers, how much of it is resident.  A
// query that fails is answered with its error and asked again the next time; devices past the last
// slot are asked every time.
class PerDevice {
 public:
  // query(int* value) returns an error code, 0 for success.
  template <class Query>
  auto get(int device, int* value, Query query) -> decltype(query(value)) {
    const bool slot = device >= 0 && device < kSlots;
    *value = slot ? kept_[device].load(std::memory_order_relaxed) : 0;
    if (*value > 0) return {};
    const auto error = query(value);
    if (slot && error == decltype(query(value)){}) kept_[device].store(*value, std::memory_order_relaxed);
    return error;
  }

 private:
  static constexpr int kSlots = 64;
  std::atomic<int> kept_[kSlots] = {};
};

}  // namespace flexq
