// Definitions of the selectors in dyt_rms_select.cuh.
#pragma once

#include "dyt_rms_select.cuh"

namespace dyt {
namespace norm {

template <typename T, bool RAGGED, bool RES, bool Q>
RmsFwdKernel rms_fwd_ring_of(const host::RowPlan &p) {
  constexpr int E = fwd_elems<T>(), EN = kNarrowElems;
  if (p.cluster) return rms_fwd_kernel<T, E, kCluster, RAGGED, RES, Q>;
  if (p.group) return rms_fwd_kernel<T, E, kGroup, RAGGED, RES, Q>;
  if (p.L == 32)
    return p.NV * p.V > 32 * EN ? rms_fwd_kernel<T, E, kWarp, RAGGED, RES, Q>
                                : rms_fwd_kernel<T, EN, kWarp, RAGGED, RES, Q>;
  return p.L == 16 ? rms_fwd_kernel<T, EN, kHalf, RAGGED, RES, Q> : rms_fwd_kernel<T, EN, kPart, RAGGED, RES, Q>;
}
template <typename T, bool RES, bool Q>
RmsFwdKernel rms_fwd_of(const host::RowPlan &p) {
  constexpr int V = 16 / (int)sizeof(T);
  if (p.rowlong) return p.V == 1 ? rms_fwd_long_kernel<T, 1, RES, Q> : rms_fwd_long_kernel<T, V, RES, Q>;
  return p.ragged ? rms_fwd_ring_of<T, true, RES, Q>(p) : rms_fwd_ring_of<T, false, RES, Q>(p);
}
template <typename T>
RmsFwdKernel rms_fwd_kernel_of(const host::RowPlan &p, bool res, bool q8) {
  if (q8) return res ? rms_fwd_of<T, true, true>(p) : rms_fwd_of<T, false, true>(p);
  return res ? rms_fwd_of<T, true, false>(p) : rms_fwd_of<T, false, false>(p);
}

template <typename T, bool RES>
RmsBwdKernel rms_bwd_of(const host::RowPlan &p) {
  if (p.cluster)
    return p.ragged ? rms_bwd_kernel<T, kClusterRows, true, RES> : rms_bwd_kernel<T, kClusterRows, false, RES>;
  if (p.group) return p.ragged ? rms_bwd_kernel<T, kGroup, true, RES> : rms_bwd_kernel<T, kGroup, false, RES>;
  if (p.L == 32) return p.ragged ? rms_bwd_kernel<T, kWarp, true, RES> : rms_bwd_kernel<T, kWarp, false, RES>;
  if (p.L == 16) return p.ragged ? rms_bwd_kernel<T, kHalf, true, RES> : rms_bwd_kernel<T, kHalf, false, RES>;
  return p.ragged ? rms_bwd_kernel<T, kPart, true, RES> : rms_bwd_kernel<T, kPart, false, RES>;
}
template <typename T>
RmsBwdKernel rms_bwd_kernel_of(const host::RowPlan &p, bool res) {
  return res ? rms_bwd_of<T, true>(p) : rms_bwd_of<T, false>(p);
}
template <typename T>
RmsBwdLongKernel rms_bwd_rows_kernel_of(const host::RowPlan &p) {
  return p.V == 1 ? rms_bwd_rows_kernel<T, 1> : rms_bwd_rows_kernel<T, 16 / (int)sizeof(T)>;
}
template <typename T>
RmsBwdColumnsKernel rms_bwd_columns_kernel_of(const host::RowPlan &p, bool res) {
  constexpr int V = 16 / (int)sizeof(T);
  if (p.V == 1) return res ? rms_bwd_columns_kernel<T, 1, true> : rms_bwd_columns_kernel<T, 1, false>;
  return res ? rms_bwd_columns_kernel<T, V, true> : rms_bwd_columns_kernel<T, V, false>;
}

#define DYT_INSTANTIATE_RMS(T)                                                            \
  template RmsFwdKernel rms_fwd_kernel_of<T>(const host::RowPlan &, bool, bool);           \
  template RmsBwdKernel rms_bwd_kernel_of<T>(const host::RowPlan &, bool);                 \
  template RmsBwdLongKernel rms_bwd_rows_kernel_of<T>(const host::RowPlan &);              \
  template RmsBwdColumnsKernel rms_bwd_columns_kernel_of<T>(const host::RowPlan &, bool);

}  // namespace norm
}  // namespace dyt
