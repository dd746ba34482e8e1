// What is found out once for each device of the process: a function's attribute, a device's property.
#pragma once

#include <atomic>

namespace moe {

constexpr int kMaxDevices = 64;

// The value of find() for `device`, kept in `kept` (zeros at first) where it is above 0; a failure (0 or
// below) is tried again by the next call.  Threads that come first together may each call find().
template <typename F>
int once_a_device(std::atomic<int> (&kept)[kMaxDevices], int device, F find) {
  if (device < 0 || device >= kMaxDevices) return find();
  int v = kept[device].load(std::memory_order_acquire);
  if (v <= 0 && (v = find()) > 0) kept[device].store(v, std::memory_order_release);
  return v;
}

}  // namespace moe
