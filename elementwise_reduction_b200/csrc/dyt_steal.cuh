// Work that goes to whoever is free: a CTA takes the place of one of its grid that has not been launched yet
// (cluster launch control). A grid of a CTA for each row then costs no more launches than fit on the SMs, and
// every SM gets as many rows as it has time for. Measured on two inputs and two outputs of 134 MB each, rows of 8
// KB: 82 us, with a fixed share of the rows for each CTA 90 (537 MB each: 315 and 354): the SMs do not get the
// same share of the memory's rate.
#pragma once

#include <cstdint>

namespace dyt {

// In shared memory. One thread initialises it and asks, all threads of the CTA take the answer; the next question
// comes after a barrier behind the last taking.
struct Steal {
  static constexpr int64_t kLost = -2;     // the wait ran out of its limit
  static constexpr int kPolls = 1 << 20;   // each waits for a while itself
  uint4 answer;
  unsigned long long bar;

  __device__ __forceinline__ uint32_t bar_at() const { return (uint32_t)__cvta_generic_to_shared(&bar); }
  __device__ __forceinline__ void init() {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar_at()) : "memory");
  }
  // (what was read of the last answer, or written to the barrier, comes before the copy of the next)
  __device__ __forceinline__ void ask() {
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(&answer);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 16;" ::"r"(bar_at()) : "memory");
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(a),
        "r"(bar_at())
        : "memory");
  }
  // The index of the CTA whose work is now this one's; -1: none is left (then nothing more may be asked).
  // phase: 0 for the first answer, then 1, 0, ...
  template <int POLLS = kPolls>
  __device__ __forceinline__ int64_t take(uint32_t phase) const {
    uint32_t done = 0;
    for (int i = 0; i < POLLS && !done; ++i)
      asm volatile("{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
                   : "=r"(done)
                   : "r"(bar_at()), "r"(phase)
                   : "memory");
    if (!done) return kLost;
    uint32_t got, x;
    asm volatile(
        "{.reg .pred p; .reg .b128 q; ld.shared.b128 q, [%2];"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, q; selp.u32 %0, 1, 0, p; mov.u32 %1, 0;"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, q;}"
        : "=r"(got), "=r"(x)
        : "r"((uint32_t)__cvta_generic_to_shared(&answer))
        : "memory");
    return got ? (int64_t)x : -1;
  }
};

}  // namespace dyt
