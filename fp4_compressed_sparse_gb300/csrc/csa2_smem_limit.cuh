// csa2_smem_limit.cuh -- the kernels' dynamic shared-memory limits as they have been raised
// so far (host code without CUDA calls of its own).
#pragma once

#include <map>
#include <mutex>
#include <utility>

namespace csa2 {

class SmemLimits {
 public:
  // Calls set(), which is to make `bytes` the limit of kernel fn on device dev, unless the limit
  // is that high already; a failure (anything but 0) is returned and not remembered.  The lock is
  // held across set(): with two threads in it at once the smaller size could be set last, below
  // the larger one that is remembered.
  template <class Set>
  auto raise(int dev, const void *fn, int bytes, Set set) -> decltype(set()) {
    std::lock_guard<std::mutex> lock(mu_);
    int &have = limit_[std::make_pair(dev, fn)];
    if (have >= bytes) return decltype(set()){};
    const auto e = set();
    if (e == decltype(e){}) have = bytes;
    return e;
  }

 private:
  std::mutex mu_;
  std::map<std::pair<int, const void *>, int> limit_;
};

}  // namespace csa2
