// The dynamic shared memory that a kernel may be launched with is an attribute
// that a call sets, not raises: two host threads that each compare, set and note
// it by themselves can leave it below what one of them noted, and every later
// launch in between fails.  Here it only grows, one thread at a time.
#pragma once

#include <atomic>
#include <mutex>

namespace pd {

class SmemLimit {
 public:
  static constexpr int kDevices = 64;

  // At least `bytes` on device dev (below kDevices): set(bytes) where no call set
  // as many before; its error, 0 for none.
  template <typename Set>
  auto raise(int dev, int bytes, Set &&set) -> decltype(set(bytes)) {
    using E = decltype(set(bytes));
    if (bytes <= set_[dev].load(std::memory_order_acquire)) return E{};
    std::lock_guard<std::mutex> lock(mu_);
    if (bytes <= set_[dev].load(std::memory_order_relaxed)) return E{};
    const E e = set(bytes);
    if (e == E{}) set_[dev].store(bytes, std::memory_order_release);
    return e;
  }

 private:
  std::mutex mu_;
  std::atomic<int> set_[kDevices] = {};
};

}  // namespace pd
