// Layer norm entry points (declared in include/dyt.h): argument checks, launch
// plans and dispatch of the kernels in dyt_norm.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dyt.h"
#include "dyt_host.h"
#include "dyt_norm.cuh"

namespace {

using namespace dyt::host;
using dyt::norm::NormArgs;
using dyt::norm::NormGradArgs;

constexpr int kOpNormForward = 5, kOpNormBackward = 6;  // dyt_launch_info::op

// How a row is spread over lanes (see dyt_norm.cuh).
struct RowPlan {
  int V = 1, L = 1, NV = 0;
  int block = 0;         // threads of a CTA
  int rows = 1;          // rows side by side in a CTA
  bool group = false;    // a row takes several warps
  bool ragged = false;   // rows off 16-byte boundaries, or of no whole vectors
  bool rowlong = false;  // too long for a CTA's registers
};

int pow2_at_least(int64_t v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// vec: elements of 16 bytes. aligned: every row of every tensor is whole aligned vectors. E: elements a lane holds.
RowPlan plan_rows(int64_t M, int64_t N, int vec, bool aligned, int E, int sms) {
  RowPlan p;
  const int64_t lanes = aligned ? ceil_div(N / vec, E / vec) : ceil_div(N, E);
  p.ragged = !aligned;
  if (lanes > dyt::norm::kBlock) {
    p.rowlong = true;
    p.V = aligned ? vec : 1;
    p.NV = (int)ceil_div(N, p.V);
    p.block = p.L = 1024;
    return p;
  }
  p.V = aligned ? vec : 1;
  p.NV = (int)ceil_div(N, p.V);
  p.group = lanes > 32;
  p.L = p.group ? (int)ceil_div(lanes, 32) * 32 : pow2_at_least(lanes);
  // Ragged rows keep one slot more per row and warp: half the threads where that is up to half a slot per lane.
  int block = p.ragged && p.L < 8 ? dyt::norm::kBlock / 2 : dyt::norm::kBlock;
  // Few short rows: smaller CTAs, so that more SMs take part.
  while (!p.group && block > 128 && ceil_div(M, block / p.L) < sms) block >>= 1;
  p.rows = block / p.L;
  p.block = p.rows * p.L;
  return p;
}

// The walk of `grid` CTAs over the rows of tensors with pitches lds (the inputs, then the output).
dyt::norm::Walk walk_of(const RowPlan &p, int64_t M, int64_t N, int64_t grid, const int64_t *lds, int n, size_t elem,
                        int plane_slots) {
  dyt::norm::Walk w = {};
  w.M = M;
  w.N = N;
  w.NV = p.NV;
  w.L = p.L;
  w.rows = p.rows;
  w.step = (int)(grid * p.rows);
  for (int i = 0; i < n; ++i) w.inc[i] = (int64_t)w.step * lds[i] * (int64_t)elem;
  // Rows at the tensors' ends whose chunks could reach past them: those less
  // than 16 bytes from the first or the last row.
  if (p.ragged)
    for (int i = 0; i + 1 < n; ++i) w.fast = std::max(w.fast, ceil_div(16, std::max<int64_t>(1, lds[i] * (int64_t)elem)));
  w.plane = plane_slots * 16;
  w.n = (float)N;
  w.inv_n = 1.0f / (float)N;
  return w;
}

template <typename T>
constexpr int vec_elems() {
  return 16 / (int)sizeof(T);
}

template <typename F>
dyt_status with_type(int xd, F &&f) {
  switch (xd) {
    case DYT_F32: return f(float{});
    case DYT_BF16: return f(__nv_bfloat16{});
    case DYT_F16: return f(__half{});
  }
  return DYT_ERR_UNSUPPORTED_DTYPE;
}

using FwdKernel = void (*)(NormArgs);
using BwdKernel = void (*)(NormGradArgs);

template <typename T>
FwdKernel fwd_kernel(const RowPlan &p) {
  using namespace dyt::norm;
  if (p.rowlong) return p.V == 1 ? norm_fwd_long_kernel<T, 1> : norm_fwd_long_kernel<T, vec_elems<T>()>;
  if (p.group) return p.ragged ? norm_fwd_kernel<T, kGroup, true> : norm_fwd_kernel<T, kGroup, false>;
  if (p.L == 32) return p.ragged ? norm_fwd_kernel<T, kWarp, true> : norm_fwd_kernel<T, kWarp, false>;
  return p.ragged ? norm_fwd_kernel<T, kPart, true> : norm_fwd_kernel<T, kPart, false>;
}
template <typename T>
BwdKernel bwd_kernel(const RowPlan &p) {
  using namespace dyt::norm;
  if (p.group) return p.ragged ? norm_bwd_kernel<T, kGroup, true> : norm_bwd_kernel<T, kGroup, false>;
  if (p.L == 32) return p.ragged ? norm_bwd_kernel<T, kWarp, true> : norm_bwd_kernel<T, kWarp, false>;
  return p.ragged ? norm_bwd_kernel<T, kPart, true> : norm_bwd_kernel<T, kPart, false>;
}

constexpr int kColumnsBlock = 256;  // vector-columns of a CTA in the long rows' second pass

// Partial sums of a backward: one set per CTA (per row group for long rows).
struct BwdPlan {
  RowPlan r;
  int64_t grid = 0;   // CTAs (the row pass's for long rows)
  int64_t parts = 0;  // partial sets
  int col_ctas = 0;   // long rows: CTAs across the columns
  size_t off_c12 = 0, bytes = 0;
};

BwdPlan plan_bwd(int64_t M, int64_t N, int vec, bool aligned, int sms) {
  BwdPlan b;
  b.r = plan_rows(M, N, vec, aligned, dyt::norm::kBwdElems, sms);
  if (b.r.rowlong) {
    b.grid = std::min<int64_t>(M, (int64_t)sms * 2);
    b.col_ctas = (int)ceil_div(b.r.NV, kColumnsBlock);
    b.parts = std::max<int64_t>(1, std::min<int64_t>(M, (int64_t)sms * 4 / b.col_ctas));
  } else {
    b.grid = std::min<int64_t>(ceil_div(M, b.r.rows), (int64_t)sms);
    b.parts = b.grid;
  }
  b.off_c12 = ((size_t)b.parts * 2 * (size_t)N * sizeof(double) + 15) & ~(size_t)15;
  b.bytes = b.off_c12 + (b.r.rowlong ? (size_t)M * sizeof(float2) : 0);
  b.bytes = (b.bytes + 15) & ~(size_t)15;
  return b;
}

void record(int op, const RowPlan *p, int64_t grid, int kernels, int64_t groups, size_t ws) {
  dyt_launch_info i = {};
  i.op = op;
  i.kernels = kernels;
  i.workspace_bytes = (int64_t)ws;
  if (p) {
    i.path = p->group || p->rowlong ? 2 : 1;
    i.vec = p->V;
    i.block = p->block;
    i.grid = (int)grid;
    i.row_lanes = p->rows;
    i.rows_per_step = p->rows;
    i.col_chunks = 1;
    i.row_groups = (int)groups;
    i.pack_rows = 1;
    i.shifted = p->ragged && !p->rowlong;
  }
  record_info(i);
}

bool param_ok(const void *p, int dt) { return p == nullptr || elem_aligned(p, dsize(dt)); }

}  // namespace

extern "C" {

dyt_status dyt_layer_norm_forward(const void *x, int64_t ldx, const void *gamma, const void *beta, float eps, void *y,
                                  int64_t ldy, float *mean, float *rstd, int64_t M, int64_t N, dyt_dtype x_dtype,
                                  dyt_dtype gamma_dtype, dyt_dtype beta_dtype, dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, x_dtype);
  if (st != DYT_OK) return st;
  if (!valid_dtype(gamma_dtype) || !valid_dtype(beta_dtype)) return DYT_ERR_UNSUPPORTED_DTYPE;
  if (!(eps >= 0.0f) || std::isinf(eps)) return DYT_ERR_INVALID_VALUE;
  if (check_pitch(M, N, ldx) != DYT_OK || check_pitch(M, N, ldy) != DYT_OK) return DYT_ERR_INVALID_VALUE;
  if (M == 1) ldx = ldy = N;  // one row has no pitch
  if (M == 0 || N == 0) {
    record(kOpNormForward, nullptr, 0, 0, 0, 0);
    return DYT_OK;
  }
  const size_t es = dsize(x_dtype);
  if (!x || !y || !elem_aligned(x, es) || !elem_aligned(y, es) || !param_ok(gamma, gamma_dtype) ||
      !param_ok(beta, beta_dtype) || !param_ok(mean, DYT_F32) || !param_ok(rstd, DYT_F32))
    return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  return with_type(x_dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    constexpr int VE = vec_elems<T>();
    const bool vec = N % VE == 0 && aligned16(x) && aligned16(y) && vec_pitch(ldx, es) && vec_pitch(ldy, es);
    const RowPlan p = plan_rows(M, N, VE, vec, dyt::norm::fwd_elems<T>(), sms);
    const FwdKernel k = fwd_kernel<T>(p);
    const size_t smem = p.rowlong ? 0 : dyt::norm::fwd_smem<T>(p.block, p.L, p.ragged);
    const dyt_status s = prepare_smem(dev, (const void *)k, (int)smem);
    if (s != DYT_OK) return s;
    const int64_t grid = std::min<int64_t>(ceil_div(M, p.rows), (int64_t)sms);
    const int64_t lds[2] = {ldx, ldy};
    NormArgs a = {x, ldx, gamma, beta, y, ldy, mean, rstd, (int)gamma_dtype, (int)beta_dtype, eps, {}};
    a.w = walk_of(p, M, N, grid, lds, 2, es, p.rowlong ? 0 : dyt::norm::fwd_plane<T>(32, p.L, p.ragged));
    PdlConfig lc((unsigned)grid, p.block, smem, (cudaStream_t)stream);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, k, a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpNormForward, &p, grid, 1, 0, 0);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);  // the host ran out of memory for the per-device facts
}

size_t dyt_layer_norm_backward_workspace_bytes(int64_t M, int64_t N, dyt_dtype x_dtype) try {
  if (check_shape(M, N, x_dtype) != DYT_OK || M == 0 || N == 0) return 0;
  int dev = 0, sms = 0;
  if (current_sms(&dev, &sms) != DYT_OK) return 0;
  const int v = 16 / (int)dsize(x_dtype);
  return std::max(plan_bwd(M, N, v, false, sms).bytes, plan_bwd(M, N, v, true, sms).bytes);
} catch (...) {
  return 0;
}

dyt_status dyt_layer_norm_backward(const void *x, int64_t ldx, const void *dy, int64_t lddy, const void *gamma,
                                   const float *mean, const float *rstd, void *dx, int64_t lddx, void *dgamma,
                                   void *dbeta, int64_t M, int64_t N, dyt_dtype x_dtype, dyt_dtype gamma_dtype,
                                   dyt_dtype beta_dtype, void *workspace, size_t workspace_bytes,
                                   dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, x_dtype);
  if (st != DYT_OK) return st;
  if (!valid_dtype(gamma_dtype) || !valid_dtype(beta_dtype)) return DYT_ERR_UNSUPPORTED_DTYPE;
  if (check_pitch(M, N, ldx) != DYT_OK || check_pitch(M, N, lddy) != DYT_OK || check_pitch(M, N, lddx) != DYT_OK)
    return DYT_ERR_INVALID_VALUE;
  if (!param_ok(dgamma, gamma_dtype) || !param_ok(dbeta, beta_dtype)) return DYT_ERR_INVALID_VALUE;
  if (M == 1) ldx = lddy = lddx = N;  // one row has no pitch
  const cudaStream_t s = (cudaStream_t)stream;
  if (M == 0 || N == 0) {
    cudaError_t e = cudaSuccess;  // empty sums
    if (N > 0 && dgamma) e = cudaMemsetAsync(dgamma, 0, (size_t)N * dsize(gamma_dtype), s);
    if (N > 0 && dbeta && e == cudaSuccess) e = cudaMemsetAsync(dbeta, 0, (size_t)N * dsize(beta_dtype), s);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpNormBackward, nullptr, 0, 0, 0, 0);
    return DYT_OK;
  }
  const size_t es = dsize(x_dtype);
  if (!x || !dy || !dx || !mean || !rstd || !workspace || !aligned16(workspace) || !elem_aligned(x, es) ||
      !elem_aligned(dy, es) || !elem_aligned(dx, es) || !param_ok(gamma, gamma_dtype) || !param_ok(mean, DYT_F32) ||
      !param_ok(rstd, DYT_F32))
    return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  return with_type(x_dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    constexpr int VE = vec_elems<T>();
    const bool vec = N % VE == 0 && aligned16(x) && aligned16(dy) && aligned16(dx) &&
                     vec_pitch(ldx, es) && vec_pitch(lddy, es) && vec_pitch(lddx, es);
    const BwdPlan b = plan_bwd(M, N, VE, vec, sms);
    if (workspace_bytes < b.bytes) return DYT_ERR_WORKSPACE_TOO_SMALL;
    double *parts = (double *)workspace;
    const int64_t lds[3] = {ldx, lddy, lddx};
    NormGradArgs a = {x, ldx, dy, lddy, gamma, mean, rstd, dx, lddx, parts, (int)gamma_dtype, {}};
    a.w = walk_of(b.r, M, N, b.grid, lds, 3, es,
                  b.r.rowlong ? 0 : dyt::norm::row_slots<T, dyt::norm::kBwdElems>(32, b.r.L, b.r.ragged));
    int kernels = 2;
    cudaError_t e;
    if (b.r.rowlong) {
      float2 *c12 = (float2 *)((char *)workspace + b.off_c12);
      PdlConfig lr((unsigned)b.grid, 1024, 0, s);
      e = cudaLaunchKernelEx(&lr.cfg, vec ? dyt::norm::norm_bwd_rows_kernel<T, VE> : dyt::norm::norm_bwd_rows_kernel<T, 1>,
                             a, c12);
      if (e != cudaSuccess) return cuda_fail(e);
      PdlConfig lc((unsigned)b.col_ctas, kColumnsBlock, 0, s);
      lc.cfg.gridDim.y = (unsigned)b.parts;
      e = cudaLaunchKernelEx(&lc.cfg,
                             vec ? dyt::norm::norm_bwd_columns_kernel<T, VE> : dyt::norm::norm_bwd_columns_kernel<T, 1>,
                             a, (const float2 *)c12);
      kernels = 3;
    } else {
      const BwdKernel k = bwd_kernel<T>(b.r);
      const size_t smem = dyt::norm::bwd_smem<T>(b.r.block, b.r.L, b.r.ragged);
      const dyt_status ready = prepare_smem(dev, (const void *)k, (int)smem);
      if (ready != DYT_OK) return ready;
      PdlConfig lc((unsigned)b.grid, b.r.block, smem, s);
      e = cudaLaunchKernelEx(&lc.cfg, k, a);
    }
    if (e != cudaSuccess) return cuda_fail(e);
    if (dgamma || dbeta) {
      PdlConfig lf((unsigned)ceil_div(N, dyt::norm::kSumCols), dyt::norm::kSumCols * dyt::norm::kSumLanes, 0, s);
      lf.cfg.gridDim.y = 2;
      e = cudaLaunchKernelEx(&lf.cfg, dyt::norm::norm_finalize_kernel, (const double *)parts, (int)b.parts, N, dgamma,
                             (int)gamma_dtype, dbeta, (int)beta_dtype);
      if (e != cudaSuccess) return cuda_fail(e);
    } else {
      --kernels;
    }
    record(kOpNormBackward, &b.r, b.grid, kernels, b.parts, b.bytes);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);
}

}  // extern "C"
