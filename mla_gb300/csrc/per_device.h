// What is set up once on each device: attributes of a kernel and limits that
// the runtime reports hold for the device that is current when they are set or
// asked for.  Host code without CUDA types.
#pragma once

#include <atomic>
#include <mutex>

namespace mla {

// A value for each device, made by the device's first user.  make(value)
// returns 0 for success; any other result is returned, nothing is kept and the
// device's next user tries again.  For use by several threads at once.
template <class T>
class PerDevice {
 public:
  template <class Make>
  auto get(int dev, T& value, Make&& make) -> decltype(make(value)) {
    using Result = decltype(make(value));
    if (dev < 0 || dev >= kMaxDevices) return make(value);  // (not kept)
    Slot& s = slot_[dev];
    if (!s.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!s.ready.load(std::memory_order_relaxed)) {
        const Result r = make(s.value);
        if (r != Result(0)) return r;
        s.ready.store(true, std::memory_order_release);
      }
    }
    value = s.value;
    return Result(0);
  }

 private:
  static constexpr int kMaxDevices = 64;
  struct Slot {
    std::atomic<bool> ready{false};
    T value{};
  };
  std::mutex mu_;
  Slot slot_[kMaxDevices];
};

}  // namespace mla
