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

}  // namespace moe
