// State of the host side that belongs to a device: a kernel's attributes, what fits a device
// at once.  Made by the first call on each device; any thread may come first.
#pragma once

#include <mutex>

namespace occult {

constexpr int kMaxDevices = 64;

template <typename T>
class PerDevice {
 public:
  // The state of `device` (0 .. kMaxDevices - 1), after `make` has run on it once.
  template <typename F>
  const T& get(int device, F&& make) {
    Slot& s = slots_[device];
    std::call_once(s.once, [&] { make(s.state); });
    return s.state;
  }

 private:
  struct Slot {
    std::once_flag once;
    T state{};
  };
  Slot slots_[kMaxDevices];
};

}  // namespace occult
