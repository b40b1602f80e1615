// kept.cuh — an answer of the driver that does not change while the process
// lives, asked for until it is given.
#pragma once

#include <atomic>

namespace cce {

// ask(&value) says whether it succeeded; only a success is kept.
class Kept {
 public:
  template <typename F>
  bool get(F ask, int* value) {
    int v = value_.load(std::memory_order_relaxed);
    if (v == kNone) {
      if (!ask(&v)) return false;
      value_.store(v, std::memory_order_relaxed);
    }
    *value = v;
    return true;
  }

 private:
  static constexpr int kNone = -1;
  std::atomic<int> value_{kNone};
};

}  // namespace cce
