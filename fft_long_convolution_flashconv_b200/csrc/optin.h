// A per-device limit that launches of one kernel raise as they need it (plain
// C++, so that it can be tested without a GPU).
#pragma once

#include <stddef.h>

#include <atomic>
#include <map>
#include <mutex>

namespace fc {

// raise(device, bytes, set) calls set(bytes) (status, 0 = done) unless the
// device's limit is that high already.  Host threads may ask for different sizes
// at once: one sets at a time, and none ever lowers what another has set.
class RaisedLimit {
 public:
  template <typename Set>
  auto raise(int device, size_t bytes, Set set) -> decltype(set(bytes)) {
    const bool known = device >= 0 && device < kKnown;
    if (known && bytes <= limit_[device].load(std::memory_order_acquire)) return {};
    const std::lock_guard<std::mutex> hold(mutex_);
    const size_t now = known ? limit_[device].load(std::memory_order_relaxed) : other_[device];
    if (bytes <= now) return {};
    const auto status = set(bytes);
    if (status == decltype(status){}) {
      if (known)
        limit_[device].store(bytes, std::memory_order_release);
      else
        other_[device] = bytes;
    }
    return status;
  }

 private:
  static constexpr int kKnown = 64;  // ordinals that are looked up without the lock
  std::atomic<size_t> limit_[kKnown] = {};
  std::map<int, size_t> other_;
  std::mutex mutex_;
};

}  // namespace fc
