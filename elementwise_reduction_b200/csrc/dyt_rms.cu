// Root-mean-square norm entry points (declared in include/dyt.h): argument
// checks, launch plans and dispatch of the kernels in dyt_rms.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dyt.h"
#include "dyt_host.h"
#include "dyt_rms_select.cuh"
#include "dyt_rows.h"

namespace {

using namespace dyt::host;
using namespace dyt::norm::host;
using dyt::norm::RmsArgs;
using dyt::norm::RmsGradArgs;
using dyt::norm::Walk;

constexpr int kOpRmsForward = 9, kOpRmsQuantize = 10, kOpRmsBackward = 11;  // dyt_launch_info::op
constexpr int kColumnsBlock = 256;  // vector-columns of a CTA in the long rows' second pass

struct FwdPlan {
  RowPlan r;
  bool narrow;    // kNarrowElems elements a lane
  bool steal;
  int64_t items;  // a CTA's or a cluster's rows of a step
  int64_t grid;
};

// Work is taken from CTAs that do not run yet where every CTA has more than kFewSteps items: the first answers cost
// 0.3 us, fixed shares the difference between the SMs. Measured with a residual, fixed and taken: 1184 x 4096 bf16
// (2 steps) 6.1 and 6.5 us, 2368 x 4096 14.0 and 14.1, 4736 x 4096 27.4 and 25.8, 9472 x 4096 56.1 and 48.2. Narrow
// rows, more of a CTA's time at its ends, gain from the second step on: 9472 x 256 5.3 and 4.5, 18944 x 256 7.1 and
// 6.5.
constexpr int kFewSteps = 4;
// Of an SM. (As the registers of half of these kernels allow; the others have 4 or 5 at once: where there are more CTAs
// than run, work is taken from those that wait, so that the number only says from when on.)
constexpr int kNarrowCtas = 6;

// Rows too long for one CTA's registers, and not for four CTAs', are shared by a cluster of 2, 4 or 8 CTAs. A step
// takes a cluster as long whatever its lanes (1.1 us), so as many threads of the device as can be have a row: `side`
// (backward): rows side by side fill the CTAs of larger clusters. (In the forward they gain up to 6% at some widths and
// lose 5 at others, by their registers.) Measured in the backward, bf16 with a residual, 4096 rows, clusters
// of 2, 4 and 8: 9216 columns 60, 54 and -, 12288 69, 75 and -, 20480 -, 137 and 121, 32768 -, 174 and 188. (Clusters
// of 3, 5, 6 or 7 take between these times and twice as long: not all that should fit run at once.)
void plan_cluster(RowPlan &p, int64_t M, int64_t N, int E, int sms, bool side) {
  if (!p.rowlong || N > (int64_t)4 * dyt::norm::kBlock * E) return;
  constexpr int kSizes[] = {2, 4, 8}, kReached[] = {74, 66, 60};  // parts of 74 of the SMs that run such clusters
  int64_t most = 0;
  for (int i = 0; i < (side ? 3 : 2); ++i) {
    const int c = kSizes[i], L = (int)ceil_div(ceil_div(N, c), 32 * E) * 32;
    if (L > dyt::norm::kBlock) continue;
    const int64_t room = side ? std::min(dyt::norm::kBlock / L, dyt::norm::kClusterMost) : 1;
    const int64_t rows = std::max<int64_t>(1, std::min(room, ceil_div(M, std::max(1, sms / c))));
    if (rows * L * kReached[i] <= most) continue;
    most = rows * L * kReached[i];
    p.cluster = c;
    p.L = L;
    p.rows = (int)rows;
    p.block = (int)rows * L;
  }
  p.rowlong = false;
  p.group = true;
  // (whole vectors and scales; the last CTA has some too, with more than 8 x 7 x kScaleCols columns)
  p.cols = (int)ceil_div(ceil_div(N, p.cluster), dyt::norm::kScaleCols) * dyt::norm::kScaleCols;
}

FwdPlan plan_fwd(int64_t M, int64_t N, int vec, bool aligned, int E, int sms) {
  FwdPlan p = {};
  p.narrow = N <= 32 * dyt::norm::kNarrowElems;
  p.r = plan_rows(M, N, vec, aligned, p.narrow ? dyt::norm::kNarrowElems : E, sms);
  plan_cluster(p.r, M, N, E, sms, false);
  p.items = M;
  p.grid = std::min<int64_t>(M, (int64_t)sms * 2);  // (long rows)
  if (p.r.rowlong || p.r.cluster) return p;
  p.r.rows = p.r.group ? 1 : dyt::norm::kNarrowBlock / p.r.L;
  p.r.block = p.r.rows * p.r.L;
  p.items = ceil_div(M, p.r.rows);
  const int64_t at_once = (int64_t)sms * (p.narrow ? kNarrowCtas : dyt::norm::kBlock / p.r.block);
  p.steal = p.items > (p.narrow ? 1 : kFewSteps) * at_once;
  p.grid = p.steal ? p.items : std::min(p.items, at_once);
  return p;
}

// A plan for few rows spreads them over the SMs: no more rows side by side than every SM gets.
RowPlan plan_rms(int64_t M, int64_t N, int vec, bool aligned, int E, int sms) {
  RowPlan p = plan_rows(M, N, vec, aligned, E, sms);
  plan_cluster(p, M, N, E, sms, true);
  if (!p.group || p.rowlong || p.cluster) return p;
  p.rows = (int)std::max<int64_t>(1, std::min<int64_t>(p.rows, ceil_div(M, sms)));
  p.block = p.rows * p.L;
  return p;
}

struct BwdPlan {
  RowPlan r;
  int64_t grid = 0;   // CTAs (the row pass's for long rows)
  int64_t parts = 0;  // partial sets
  int col_ctas = 0;   // long rows: CTAs across the columns
  size_t off_c = 0, bytes = 0;
};

// Few rows, one or two steps of a CTA, are one CTA's, whose column sums need no others: a launch less, and no
// workspace. Measured, with a CTA for each row or few and in one CTA: the call, by the host, 16.6 and 12.0 us; the
// kernels, bf16 with a residual, 1 x 4096 5.8 and 4.6, 4 x 4096 (two steps) 5.9 and 6.4, 40 x 255 binary32 (two) 4.9
// and 6.2; three steps, 6 x 4096 6.1 and 7.3, 300 x 64 binary32 5.9 and 9.0.
constexpr int kOneCtaSteps = 2;
int one_cta_rows(const RowPlan &p) { return (p.ragged && p.L < 8 ? dyt::norm::kBlock / 2 : dyt::norm::kBlock) / p.L; }

BwdPlan plan_bwd(int64_t M, int64_t N, int vec, bool aligned, int sms) {
  BwdPlan b;
  b.r = plan_rms(M, N, vec, aligned, dyt::norm::kBwdElems, sms);
  if (b.r.rowlong) {
    b.grid = std::min<int64_t>(M, (int64_t)sms * 2);
    b.col_ctas = (int)ceil_div(b.r.NV, kColumnsBlock);
    b.parts = std::max<int64_t>(1, std::min<int64_t>(M, (int64_t)sms * 4 / b.col_ctas));
  } else if (!b.r.cluster && ceil_div(M, one_cta_rows(b.r)) <= kOneCtaSteps) {
    const int side = b.r.L < 32 ? 32 / b.r.L : 1;  // rows of a warp
    b.r.rows = (int)std::min<int64_t>(one_cta_rows(b.r), ceil_div(M, side) * side);
    b.r.block = b.r.rows * b.r.L;
    b.grid = 1;
    return b;
  } else {
    // (of clusters at most as many: the launch knows how many fit)
    b.grid = std::min<int64_t>(ceil_div(M, b.r.rows), (int64_t)(b.r.cluster ? std::max(1, sms / b.r.cluster) : sms));
    b.parts = b.grid;
  }
  b.off_c = ((size_t)b.parts * (size_t)N * sizeof(double) + 15) & ~(size_t)15;
  b.bytes = b.off_c + (b.r.rowlong ? (size_t)M * sizeof(float) : 0);
  b.bytes = (b.bytes + 15) & ~(size_t)15;
  return b;
}

// The workspace, whatever the rows' alignment.
size_t most_bytes(int64_t M, int64_t N, size_t es, int sms) {
  const int v = 16 / (int)es;
  return std::max(plan_bwd(M, N, v, false, sms).bytes, plan_bwd(M, N, v, true, sms).bytes);
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
    i.col_chunks = p->cluster ? p->cluster : 1;
    i.row_groups = (int)groups;
    i.pack_rows = 1;
    i.shifted = p->ragged && !p->rowlong;
  }
  record_info(i);
}

// The launch of as many of a plan's clusters as there are rows, or as run at once.
dyt_status fit_clusters(int dev, const void *kernel, const RowPlan &r, int64_t M, int sms, PdlConfig &lc,
                        int64_t *clusters) {
  int n = 0;
  lc.cluster((unsigned)r.cluster);
  lc.cfg.gridDim.x = (unsigned)r.cluster;  // (the question is of whole clusters)
  const dyt_status st = cluster_capacity(dev, kernel, lc.cfg, r.cluster, &n);
  if (st != DYT_OK) return st;
  *clusters = std::min<int64_t>(ceil_div(M, r.rows), std::min(n, std::max(1, sms / r.cluster)));
  lc.cfg.gridDim.x = (unsigned)(*clusters * r.cluster);
  return DYT_OK;
}

// Both forward calls. q8: y is e4m3 bytes with scales, one a row (group 0) or one for each kScaleCols columns.
dyt_status forward(bool q8, const void *x, int64_t ldx, const void *res, int64_t ldr, const void *gamma, float eps,
                   int group, void *y, int64_t ldy, float *scale, void *h, int64_t ldh, float *rstd, int64_t M,
                   int64_t N, dyt_dtype x_dtype, dyt_dtype gamma_dtype, dyt_stream_t stream) {
  dyt_status st = check_shape(M, N, x_dtype);
  if (st != DYT_OK) return st;
  if (!valid_dtype(gamma_dtype)) return DYT_ERR_UNSUPPORTED_DTYPE;
  if (!(eps >= 0.0f) || std::isinf(eps) || (group != 0 && group != dyt::norm::kScaleCols)) return DYT_ERR_INVALID_VALUE;
  if (check_pitch(M, N, ldx) != DYT_OK || check_pitch(M, N, ldy) != DYT_OK) return DYT_ERR_INVALID_VALUE;
  if (res && (check_pitch(M, N, ldr) != DYT_OK || check_pitch(M, N, ldh) != DYT_OK)) return DYT_ERR_INVALID_VALUE;
  if (M == 1) ldx = ldr = ldy = ldh = N;  // one row has no pitch
  const int op = q8 ? kOpRmsQuantize : kOpRmsForward;
  if (M == 0 || N == 0) {
    record(op, nullptr, 0, 0, 0, 0);
    return DYT_OK;
  }
  const size_t es = dsize(x_dtype);
  if (!x || !y || (q8 && !scale) || (res && (!h || h == y)) || !elem_aligned(x, es) || !elem_aligned(res, es) ||
      (!q8 && !elem_aligned(y, es)) || (res && !elem_aligned(h, es)) || !param_ok(gamma, gamma_dtype) ||
      !param_ok(rstd, DYT_F32) || !param_ok(scale, DYT_F32))
    return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  return with_type(x_dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    constexpr int VE = vec_elems<T>();
    // an 8-bit row is whole vectors of VE bytes
    const bool out = q8 ? elem_aligned(y, VE) && (ldy & (VE - 1)) == 0 : aligned16(y) && vec_pitch(ldy, es);
    const bool vec = N % VE == 0 && out && aligned16(x) && vec_pitch(ldx, es) &&
                     (!res || (aligned16(res) && aligned16(h) && vec_pitch(ldr, es) && vec_pitch(ldh, es)));
    const FwdPlan p = plan_fwd(M, N, VE, vec, dyt::norm::fwd_elems<T>(), sms);
    const RowPlan &r = p.r;
    const bool ring = !r.rowlong;
    const dyt::norm::RmsFwdKernel k = dyt::norm::rms_fwd_kernel_of<T>(r, res != nullptr, q8);
    if (p.grid > INT32_MAX) return DYT_ERR_INVALID_VALUE;  // (more rows than any memory holds)
    constexpr int E = dyt::norm::fwd_elems<T>(), EN = dyt::norm::kNarrowElems;
    const size_t smem = !ring ? 0 : p.narrow ? dyt::norm::rms_fwd_smem<T, EN>(r.block, r.L, r.ragged, res != nullptr)
                                             : dyt::norm::rms_fwd_smem<T, E>(r.block, r.L, r.ragged, res != nullptr);
    dyt_status s = prepare_smem(dev, (const void *)k, (int)smem);
    if (s != DYT_OK) return s;
    const int64_t lds[3] = {ldx, res ? ldr : ldx, ldx};  // the inputs (walk_of takes the last for an output)
    RmsArgs a = {};
    a.x = x;
    a.ldx = ldx;
    a.res = res;
    a.ldr = ldr;
    a.gamma = gamma;
    a.y = y;
    a.ldy = ldy;
    a.h = res ? h : nullptr;
    a.ldh = ldh;
    a.rstd = rstd;
    a.scale = scale;
    a.gamma_dt = (int)gamma_dtype;
    a.eps = eps;
    a.grouped = group != 0;
    a.groups = group ? (int)ceil_div(N, group) : 1;
    a.steal = p.steal;
    a.items = p.items;
    a.w = walk_of(r, M, N, 0, lds, 3, es,
                  !ring      ? 0
                  : p.narrow ? dyt::norm::row_slots<T, EN>(32, r.L, r.ragged)
                             : dyt::norm::row_slots<T, E>(32, r.L, r.ragged));
    a.cols = r.cols;
    PdlConfig lc((unsigned)p.grid, r.block, smem, (cudaStream_t)stream);
    if (r.cluster) {
      int64_t clusters = 0;
      s = fit_clusters(dev, (const void *)k, r, M, sms, lc, &clusters);
      if (s != DYT_OK) return s;
    }
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, k, a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(op, &r, lc.cfg.gridDim.x, 1, 0, 0);
    return DYT_OK;
  });
}

}  // namespace

extern "C" {

dyt_status dyt_rms_norm_forward(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *gamma,
                                float eps, void *y, int64_t ldy, void *h, int64_t ldh, float *rstd, int64_t M,
                                int64_t N, dyt_dtype x_dtype, dyt_dtype gamma_dtype, dyt_stream_t stream) try {
  return forward(false, x, ldx, residual, ldr, gamma, eps, 0, y, ldy, nullptr, h, ldh, rstd, M, N, x_dtype,
                 gamma_dtype, stream);
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);  // the host ran out of memory for the per-device facts
}

dyt_status dyt_rms_norm_quantize(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *gamma,
                                 float eps, int group, void *q, int64_t ldq, float *scale, void *h, int64_t ldh,
                                 int64_t M, int64_t N, dyt_dtype x_dtype, dyt_dtype gamma_dtype,
                                 dyt_stream_t stream) try {
  return forward(true, x, ldx, residual, ldr, gamma, eps, group, q, ldq, scale, h, ldh, nullptr, M, N, x_dtype,
                 gamma_dtype, stream);
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);
}

size_t dyt_rms_norm_backward_workspace_bytes(int64_t M, int64_t N, dyt_dtype x_dtype) try {
  if (check_shape(M, N, x_dtype) != DYT_OK || M == 0 || N == 0) return 0;
  int dev = 0, sms = 0;
  if (current_sms(&dev, &sms) != DYT_OK) return 0;
  return std::max<size_t>(16, most_bytes(M, N, dsize(x_dtype), sms));
} catch (...) {
  return 0;
}

dyt_status dyt_rms_norm_backward(const void *h, int64_t ldh, const void *dy, int64_t lddy, const float *rstd,
                                 const void *gamma, const void *dh, int64_t lddh, void *dx, int64_t lddx,
                                 void *dgamma, int64_t M, int64_t N, dyt_dtype x_dtype, dyt_dtype gamma_dtype,
                                 void *workspace, size_t workspace_bytes, dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, x_dtype);
  if (st != DYT_OK) return st;
  if (!valid_dtype(gamma_dtype)) return DYT_ERR_UNSUPPORTED_DTYPE;
  if (check_pitch(M, N, ldh) != DYT_OK || check_pitch(M, N, lddy) != DYT_OK || check_pitch(M, N, lddx) != DYT_OK ||
      (dh && check_pitch(M, N, lddh) != DYT_OK) || !param_ok(dgamma, gamma_dtype))
    return DYT_ERR_INVALID_VALUE;
  if (M == 1) ldh = lddy = lddh = lddx = N;  // one row has no pitch
  const cudaStream_t s = (cudaStream_t)stream;
  if (M == 0 || N == 0) {
    if (N > 0 && dgamma) {  // empty sums
      const cudaError_t e = cudaMemsetAsync(dgamma, 0, (size_t)N * dsize(gamma_dtype), s);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    record(kOpRmsBackward, nullptr, 0, 0, 0, 0);
    return DYT_OK;
  }
  const size_t es = dsize(x_dtype);
  if (!h || !dy || !dx || !rstd || !aligned16(workspace) || !elem_aligned(h, es) ||
      !elem_aligned(dy, es) || !elem_aligned(dh, es) || !elem_aligned(dx, es) || !param_ok(gamma, gamma_dtype) ||
      !param_ok(rstd, DYT_F32))
    return DYT_ERR_INVALID_VALUE;
  if (!workspace && most_bytes(M, N, es, 1)) return DYT_ERR_INVALID_VALUE;  // (whether there are any: on any device)
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  return with_type(x_dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    constexpr int VE = vec_elems<T>();
    const bool res = dh != nullptr;
    const bool vec = N % VE == 0 && aligned16(h) && aligned16(dy) && aligned16(dh) && aligned16(dx) &&
                     vec_pitch(ldh, es) && vec_pitch(lddy, es) && vec_pitch(lddx, es) && (!res || vec_pitch(lddh, es));
    const BwdPlan b = plan_bwd(M, N, VE, vec, sms);
    if (workspace_bytes < b.bytes) return DYT_ERR_WORKSPACE_TOO_SMALL;
    double *parts = b.bytes ? (double *)workspace : nullptr;
    const int64_t lds[4] = {ldh, lddy, res ? lddh : lddy, lddx};
    RmsGradArgs a = {};
    a.h = h;
    a.ldh = ldh;
    a.dy = dy;
    a.lddy = lddy;
    a.dres = dh;
    a.lddr = lddh;
    a.gamma = gamma;
    a.rstd = rstd;
    a.dx = dx;
    a.lddx = lddx;
    a.parts = parts;
    a.dgamma = dgamma;
    a.gamma_dt = (int)gamma_dtype;
    a.w = walk_of(b.r, M, N, b.grid, lds, 4, es,
                  b.r.rowlong ? 0 : dyt::norm::row_slots<T, dyt::norm::kBwdElems>(32, b.r.L, b.r.ragged));
    a.inc_dx = a.w.inc[3];
    int kernels = 1;
    int64_t parts_used = b.parts, ctas = b.grid;
    cudaError_t e;
    if (b.r.rowlong) {
      float *c = (float *)((char *)workspace + b.off_c);
      PdlConfig lr((unsigned)b.grid, 1024, 0, s);
      e = cudaLaunchKernelEx(&lr.cfg, dyt::norm::rms_bwd_rows_kernel_of<T>(b.r), a, c);
      if (e != cudaSuccess) return cuda_fail(e);
      PdlConfig lc((unsigned)b.col_ctas, kColumnsBlock, 0, s);
      lc.cfg.gridDim.y = (unsigned)b.parts;
      e = cudaLaunchKernelEx(&lc.cfg, dyt::norm::rms_bwd_columns_kernel_of<T>(b.r, res), a, (const float *)c);
      kernels = 2;
    } else {
      const dyt::norm::RmsBwdKernel k = dyt::norm::rms_bwd_kernel_of<T>(b.r, res);
      const size_t smem = dyt::norm::rms_bwd_smem<T>(b.r.block, b.r.L, b.r.ragged, res);
      const dyt_status ready = prepare_smem(dev, (const void *)k, (int)smem);
      if (ready != DYT_OK) return ready;
      PdlConfig lc((unsigned)b.grid, b.r.block, smem, s);
      a.cols = b.r.cols;
      if (b.r.cluster) {
        const dyt_status fit = fit_clusters(dev, (const void *)k, b.r, M, sms, lc, &parts_used);
        if (fit != DYT_OK) return fit;
        const Walk w = walk_of(b.r, M, N, parts_used, lds, 4, es, 0);
        a.w.step = w.step;
        for (int i = 0; i < 4; ++i) a.w.inc[i] = w.inc[i];
        a.inc_dx = w.inc[3];
      }
      ctas = (int64_t)lc.cfg.gridDim.x;
      e = cudaLaunchKernelEx(&lc.cfg, k, a);
    }
    if (e != cudaSuccess) return cuda_fail(e);
    if (dgamma && parts) {
      PdlConfig lf((unsigned)ceil_div(N, dyt::norm::kSumCols), dyt::norm::kSumCols * dyt::norm::kSumLanes, 0, s);
      e = cudaLaunchKernelEx(&lf.cfg, dyt::norm::norm_finalize_kernel<1>, (const double *)parts, (int)parts_used, N,
                             dgamma, (int)gamma_dtype, (void *)nullptr, (int)gamma_dtype);
      if (e != cudaSuccess) return cuda_fail(e);
      ++kernels;
    }
    record(kOpRmsBackward, &b.r, ctas, kernels, parts_used, b.bytes);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);
}

}  // extern "C"
