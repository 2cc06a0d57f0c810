// Counts that a device is asked for once (host side, without CUDA).
#pragma once

#include <atomic>

namespace s2 {

// A count per device and size.  What a query that succeeded gave is kept; one that
// failed is asked again at the next call.  Threads may ask at the same time.
template <int SIZES>
class KeptCounts {
 public:
  // query(int* n) returns 0 or an error, which is passed on and leaves *n alone.
  template <typename F>
  auto get(int dev, int size, int* n, F query) -> decltype(query(n)) {
    const bool keeps = dev >= 0 && dev < kDevices && size >= 0 && size < SIZES;
    if (keeps) {
      const int k = kept_[dev][size].load();
      if (k) {
        *n = k - 1;
        return {};
      }
    }
    int m = 0;
    const auto e = query(&m);
    if (e == decltype(query(n)){}) {
      *n = m;
      if (keeps) kept_[dev][size].store(m + 1);
    }
    return e;
  }

 private:
  static constexpr int kDevices = 16;
  std::atomic<int> kept_[kDevices][SIZES] = {};
};

}  // namespace s2
