// host.cuh -- host-side rules of the launches that need no GPU: plain C++, so that they are tested
// without one.
#pragma once

#include <mutex>
#include <unordered_map>

namespace moe {

// What a query said for each device and `what` (a small number).  A query that failed (an answer
// below 1) is asked again the next time.
class DeviceAnswers {
 public:
  template <typename Q>
  int get(int dev, int what, Q query) {
    const long key = (long)dev * 65536 + what;
    std::lock_guard<std::mutex> g(mu_);
    auto it = known_.find(key);
    if (it != known_.end()) return it->second;
    const int v = query();
    if (v >= 1) known_[key] = v;
    return v;
  }

 private:
  std::mutex mu_;
  std::unordered_map<long, int> known_;
};

// CTAs of a sort of n slots: a warp walks its run 32 slots at a time, so past two steps a warp of
// one CTA (1024 threads) a cluster of eight, past four steps of those sixteen.  launch(ctas) returns
// 0 when it started; a cluster of sixteen is more than every device and context must have room for
// (one that owns part of the SMs may not), so where it is refused eight do the same work.
template <typename F>
int sort_launch(long n, F launch) {
  const int ctas = n <= 1024 * 2 ? 1 : n <= 1024 * 32 ? 8 : 16;
  const int e = launch(ctas);
  return e != 0 && ctas == 16 ? launch(8) : e;
}

}  // namespace moe
