// kl_host.h -- what the library's host side keeps between calls: facts about a
// device (its SM count, its architecture, how many clusters fit on it), never
// anything of a call's data.
#pragma once

#include <atomic>

namespace kl {

constexpr int kMaxDevices = 64;

// An int per device, asked for when it is first wanted.  Host threads may call
// at once: those that find none all ask, and get and store the same answer.
// ask() does not return 0.
class DeviceValue {
 public:
  template <typename Ask>
  int get(int dev, Ask ask) {
    if (dev < 0 || dev >= kMaxDevices) return ask();  // not kept: asked every time
    int v = value_[dev].load(std::memory_order_relaxed);
    if (v == 0) {
      v = ask();
      value_[dev].store(v, std::memory_order_relaxed);
    }
    return v;
  }

 private:
  std::atomic<int> value_[kMaxDevices] = {};
};

}  // namespace kl
