// The dynamic shared memory that kernels have been opted in to, by a key for
// device and kernel. Host logic only: the CUDA call is the caller's.
#pragma once

#include <cstdint>
#include <mutex>
#include <unordered_map>

namespace dyt {
namespace host {

class SmemOptIn {
 public:
  // Has set(bytes) called unless a call for at least as many bytes has succeeded; returns its result (0: success).
  // A kernel is launched with several sizes, from several threads: look-up, call and record are one step
  // under the lock, so that a limit is only ever raised, and is in force before anyone reads it as ready.
  template <typename Set>
  int raise(uint64_t key, int bytes, Set &&set) {
    std::lock_guard<std::mutex> lk(mu_);
    auto it = ready_.find(key);
    if (it != ready_.end() && it->second >= bytes) return 0;
    const int e = set(bytes);
    if (e == 0) ready_[key] = bytes;
    return e;
  }

 private:
  std::mutex mu_;
  std::unordered_map<uint64_t, int> ready_;
};

}  // namespace host
}  // namespace dyt
