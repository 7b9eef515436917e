// A thread-block cluster whose CTAs share a row: each has a stretch of its columns, and what their warps found of
// it meets in the shared memory of all of them. Measured, 4096 x 20480 bf16 with a residual: 117 us; with the
// cluster's barrier for every row, when that was built, 149, and with one CTA that reads the row twice 207.
#pragma once

#include <cstdint>

namespace dyt {

constexpr int kMaxCluster = 8;  // CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; what each wrote before is there for the others behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// v to the place of *p in another CTA's shared memory (which has started, and does not end before a barrier).
__device__ __forceinline__ void cluster_put(float4 *p, uint32_t cta, float4 v) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile(
      "{.reg .u32 r; mapa.shared::cluster.u32 r, %0, %1; st.shared::cluster.v4.f32 [r], {%2, %3, %4, %5};}" ::"r"(at),
      "r"(cta), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
      : "memory");
}
__device__ __forceinline__ void cluster_put(float *p, uint32_t cta, float v) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("{.reg .u32 r; mapa.shared::cluster.u32 r, %0, %1; st.shared::cluster.f32 [r], %2;}" ::"r"(at), "r"(cta),
               "f"(v)
               : "memory");
}
template <typename H>
__device__ __forceinline__ void cluster_put(H *p, uint32_t cta, H v) {  // 16 bits
  static_assert(sizeof(H) == 2);
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("{.reg .u32 r; mapa.shared::cluster.u32 r, %0, %1; st.shared::cluster.u16 [r], %2;}" ::"r"(at), "r"(cta),
               "h"(*reinterpret_cast<const unsigned short *>(&v))
               : "memory");
}

// Where a row's sums of all the cluster's warps meet: each warp sends its own to every CTA (st.async) and waits for all
// of them at its CTA's mbarrier. Rows take turns between two places; a warp is at most one row ahead of another, as it
// has the other's sums of the row before. In shared memory, one for each of a CTA's rows side by side. (The norm's
// forward takes two steps for a row where its largest value meets too.)
struct Meet {
  static constexpr int kWarps = 64;       // of a row, at most
  static constexpr int kPolls = 1 << 20;  // of a wait, each waits for a while itself
  float of[2][kWarps];                    // (0 where there is no warp)
  unsigned long long bar[2];

  // Lane `lane` of the row's L in this CTA; before any put all threads of the cluster meet.
  __device__ __forceinline__ void init(int lane, int L) {
    for (int i = lane; i < 2 * kWarps; i += L) of[0][i] = 0.0f;
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar_at(i)) : "memory");
        expect(i, L);
      }
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  }
  // The warp's v (the same in all its lanes) of the row's step `it`.
  __device__ __forceinline__ void put(int it, float v, int lane, int L) {
    const uint32_t cta = lane & 31;
    if (cta >= cluster_ctas()) return;
    const int par = it & 1;
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(&of[par][((int)cluster_rank() * L + lane) / 32]);
    asm volatile(
        "{.reg .u32 r, m; mapa.shared::cluster.u32 r, %0, %2; mapa.shared::cluster.u32 m, %1, %2;"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [r], %3, [m];}" ::"r"(at),
        "r"(bar_at(par)), "r"(cta), "f"(v)
        : "memory");
  }
  // All of step `it` is in of[it & 1]; false: not within the limit. The barrier is then left as it is: its phase has
  // had the one arrival it counts, and one more before it ends is not defined.
  template <int POLLS = kPolls>
  __device__ __forceinline__ bool wait(int it, int lane, int L) {
    const int par = it & 1;
    uint32_t done = 0;
    for (int i = 0; i < POLLS && !done; ++i)
      asm volatile(
          "{.reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
          : "=r"(done)
          : "r"(bar_at(par)), "r"((uint32_t)it >> 1 & 1u)
          : "memory");
    if (done && lane == 0) expect(par, L);
    return done != 0;
  }

 private:
  __device__ __forceinline__ uint32_t bar_at(int i) const { return (uint32_t)__cvta_generic_to_shared(&bar[i]); }
  __device__ __forceinline__ void expect(int i, int L) const {
    const uint32_t bytes = cluster_ctas() * ((uint32_t)L / 32) * (uint32_t)sizeof(float);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar_at(i)), "r"(bytes) : "memory");
  }
};

}  // namespace dyt
