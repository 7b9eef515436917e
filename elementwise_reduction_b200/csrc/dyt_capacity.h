// How many clusters of a launch run at once, by all that the answer depends on.
// Host logic only: the CUDA call is the caller's.
#pragma once

#include <cstddef>
#include <map>
#include <mutex>
#include <tuple>

namespace dyt {
namespace host {

class Capacities {
 public:
  // The number that ask(&n) gave (at least 1) for this device, kernel, threads and dynamic shared memory of a CTA and
  // CTAs of a cluster; asked for once. Returns ask's error, which is not kept (0: success).
  template <typename Ask>
  int get(int dev, const void *kernel, unsigned threads, size_t smem, int ctas, int *n, Ask &&ask) {
    const Key key(dev, kernel, threads, smem, ctas);
    {
      std::lock_guard<std::mutex> lk(mu_);
      auto it = known_.find(key);
      if (it != known_.end()) {
        *n = it->second;
        return 0;
      }
    }
    int got = 0;
    const int e = ask(&got);
    if (e != 0) return e;
    *n = got < 1 ? 1 : got;
    std::lock_guard<std::mutex> lk(mu_);
    known_[key] = *n;
    return 0;
  }

 private:
  using Key = std::tuple<int, const void *, unsigned, size_t, int>;
  std::mutex mu_;
  std::map<Key, int> known_;
};

}  // namespace host
}  // namespace dyt
