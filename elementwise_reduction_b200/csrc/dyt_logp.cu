// Log probability entry points (declared in include/dyt.h): argument checks,
// launch plans and dispatch of the kernels in dyt_logp.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dyt.h"
#include "dyt_host.h"
#include "dyt_logp.cuh"
#include "dyt_loss_plan.h"

namespace {

using namespace dyt::host;
using namespace dyt::loss::host;
using dyt::loss::LogpArgs;
using dyt::loss::LogpGradArgs;

constexpr int kOpLogpForward = 12, kOpLogpBackward = 13;  // dyt_launch_info::op

struct LogpPlan {
  LossPlan p;
  int together;  // rows that a warp of logp_top_kernel takes at a time
  int cluster;   // few rows: CTAs that share one (logp_few_kernel), else 0
  int warps;     // of each
  size_t off_tops, off_taken, bytes;
};

// Few rows: one kernel, where their clusters are at most so many CTAs, 4 for each of 148 SMs. Measured, in two kernels
// and in one, bf16 with 20 alternatives: 1 x 131072 8.6 and 8.2 us, 32 x 131072 10.5 and 9.4, 64 x 131072 14.7 and
// 10.9, 256 x 32000 14.9 and 10.8, but 128 x 131072 (1024 CTAs) without alternatives 11.4 and 12.9, 512 x 32000 18.8
// and 19.5; a call by the host 20.2 and 16.2.
constexpr int kFewCtas = 592;
int few_cluster(int64_t M, int64_t N, size_t es, int *warps) {
  const int64_t batches = std::max<int64_t>(1, ceil_div(ceil_div(N * (int64_t)es, 16), dyt::loss::kBatch * 32));
  if (batches > dyt::loss::kFewBatches) return 0;
  int w = 1, c = 1;
  while (w < dyt::loss::kFewWarps && w < batches) w <<= 1;
  while (c < dyt::kMaxCluster && c * w < batches) c <<= 1;
  *warps = w;
  return M * c <= kFewCtas ? c : 0;
}

LogpPlan plan_logp(int64_t M, int64_t N, int top, size_t es, int sms) {
  LogpPlan q = {};
  q.cluster = few_cluster(M, N, es, &q.warps);
  if (q.cluster) {
    q.p.S = q.cluster * q.warps;
    q.p.block = q.warps * 32;
    q.p.grid = M * q.cluster;
    q.p.cta = true;
    q.bytes = 16;
    return q;
  }
  q.p = plan_forward(M, N, es, sms);
  if (top > 0) {
    // as many rows at a time as let the warps take them in one round
    const int64_t warps = (int64_t)sms * dyt::loss::kTopCtas * (dyt::loss::kTopBlock / 32);
    q.together = (int)std::max<int64_t>(1, std::min<int64_t>(32, ceil_div(M, warps)));
    q.p.finish = (int)std::min<int64_t>(ceil_div(M, (int64_t)q.together * (dyt::loss::kTopBlock / 32)),
                                        (int64_t)sms * dyt::loss::kTopCtas);
  }
  const size_t batches = (size_t)ceil_div(ceil_div(N * (int64_t)es, 16), dyt::loss::kBatch * 32);
  q.off_tops = ((size_t)M * (size_t)q.p.most * sizeof(float4) + 15) & ~(size_t)15;
  q.off_taken = q.off_tops + (top > 0 ? ((size_t)M * batches * 32 * es + 15) & ~(size_t)15 : 0);
  q.bytes = q.off_taken + 16;
  return q;
}

}  // namespace

extern "C" {

size_t dyt_log_probs_workspace_bytes(int64_t M, int64_t N, int top, dyt_dtype dtype) try {
  if (check_shape(M, N, dtype) != DYT_OK || M == 0 || N == 0) return 0;
  if (top < 0 || top > dyt::loss::kMaxTop || top > N) return 0;
  int dev = 0, sms = 0;
  if (current_sms(&dev, &sms) != DYT_OK) return 0;
  return plan_logp(M, N, top, dsize(dtype), sms).bytes;
} catch (...) {
  return 0;
}

dyt_status dyt_log_probs_forward(const void *logits, int64_t ld, const void *tokens, int token_bytes,
                                 int64_t ignore_index, int top, double temperature, float *logp, float *entropy,
                                 float *top_logp, int64_t *top_tokens, float *stats, int64_t M, int64_t N,
                                 dyt_dtype dtype, void *workspace, size_t workspace_bytes, dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, dtype);
  if (st != DYT_OK) return st;
  if (check_pitch(M, N, ld) != DYT_OK || (tokens && token_bytes != 4 && token_bytes != 8) || top < 0 ||
      top > dyt::loss::kMaxTop || (M > 0 && (N == 0 || top > N)) || !finite_positive(temperature))
    return DYT_ERR_INVALID_VALUE;
  if (M == 0) {
    record(kOpLogpForward, nullptr, 0, 0, 0);
    return DYT_OK;
  }
  if (M == 1) ld = N;  // one row has no pitch
  const size_t es = dsize(dtype);
  if (!logits || (tokens && !logp) || !entropy || !stats || (top > 0 && (!top_logp || !top_tokens)) ||
      !elem_aligned(logits, es) || (tokens && !elem_aligned(tokens, token_bytes)) || !elem_aligned(logp, 4) ||
      !elem_aligned(entropy, 4) || !elem_aligned(top_logp, 4) || !elem_aligned(top_tokens, 8) ||
      !elem_aligned(stats, 8) || !aligned16(workspace))
    return DYT_ERR_INVALID_VALUE;
  const float C = (float)(dyt::loss::kLog2eD / temperature);
  int warps = 0;
  if (!(C > 0.0f) || std::isinf(C) || (!workspace && !few_cluster(M, N, es, &warps))) return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  const LogpPlan q = plan_logp(M, N, top, es, sms);
  const LossPlan &p = q.p;
  if (!q.cluster && workspace_bytes < q.bytes) return DYT_ERR_WORKSPACE_TOO_SMALL;
  LogpArgs a = {};
  a.z = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.ignore = ignore_index;
  a.logp = tokens ? logp : nullptr;
  a.entropy = entropy;
  a.stats = (float2 *)stats;
  a.best = top_logp;
  a.ids = (long long *)top_tokens;
  a.parts = (float4 *)workspace;
  a.tops = (char *)workspace + q.off_tops;
  a.taken = (int *)((char *)workspace + q.off_taken);
  a.M = M;
  a.N = N;
  a.S = p.S;
  a.most = p.most;
  a.batches = (int)ceil_div(ceil_div(N * (int64_t)es, 16), dyt::loss::kBatch * 32);
  a.listed = !q.cluster && tokens != nullptr && lists_rows(p, M);
  a.aligned = N % (16 / (int64_t)es) == 0 && aligned16(logits) && vec_pitch(ld, es);
  a.wide_tokens = token_bytes == 8;
  a.K = top;
  a.together = q.together;
  a.C = C;
  a.inv_t = 1.0 / temperature;
  const cudaStream_t s = (cudaStream_t)stream;
  return with_type(dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    if (q.cluster) {
      const auto k = top > 0 ? dyt::loss::logp_few_kernel<T, true> : dyt::loss::logp_few_kernel<T, false>;
      const size_t tops = top > 0 ? (size_t)a.batches * 32 * es : 0;
      const dyt_status ready = prepare_smem(dev, (const void *)k, (int)tops);
      if (ready != DYT_OK) return ready;
      PdlConfig l((unsigned)p.grid, p.block, tops, s);
      l.cluster((unsigned)q.cluster);
      const cudaError_t e = cudaLaunchKernelEx(&l.cfg, k, a);
      if (e != cudaSuccess) return cuda_fail(e);
      record(kOpLogpForward, &p, (int)(16 / sizeof(T)), 1, 0);
      return DYT_OK;
    }
    const auto rows = top > 0 ? dyt::loss::logp_rows_kernel<T, true> : dyt::loss::logp_rows_kernel<T, false>;
    const auto finish = top > 0 ? dyt::loss::logp_top_kernel<T> : dyt::loss::logp_finish_kernel<T>;
    const size_t smem = dyt::loss::rows_smem(p.block);
    const dyt_status ready = prepare_smem(dev, (const void *)rows, (int)smem);
    if (ready != DYT_OK) return ready;
    PdlConfig lc((unsigned)p.grid, p.block, smem, s);
    cudaError_t e = cudaLaunchKernelEx(&lc.cfg, rows, a);
    if (e != cudaSuccess) return cuda_fail(e);
    PdlConfig lf((unsigned)p.finish, top > 0 ? dyt::loss::kTopBlock : dyt::loss::kFinishBlock, 0, s);
    e = cudaLaunchKernelEx(&lf.cfg, finish, a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpLogpForward, &p, (int)(16 / sizeof(T)), 2, q.bytes);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);  // the host ran out of memory for the per-device facts
}

dyt_status dyt_log_probs_backward(const void *logits, int64_t ld, const void *tokens, int token_bytes,
                                  int64_t ignore_index, const float *stats, const float *entropy,
                                  const float *grad_logp, const float *grad_entropy, double temperature,
                                  void *dlogits, int64_t lddl, int64_t M, int64_t N, dyt_dtype dtype,
                                  dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, dtype);
  if (st != DYT_OK) return st;
  if (check_pitch(M, N, ld) != DYT_OK || check_pitch(M, N, lddl) != DYT_OK ||
      (tokens && token_bytes != 4 && token_bytes != 8) || !finite_positive(temperature))
    return DYT_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) {
    record(kOpLogpBackward, nullptr, 0, 0, 0);
    return DYT_OK;
  }
  if (M == 1) ld = lddl = N;  // one row has no pitch
  const size_t es = dsize(dtype);
  if (!logits || !stats || !dlogits || (grad_logp && !tokens) || (grad_entropy && !entropy) ||
      !elem_aligned(logits, es) || (tokens && !elem_aligned(tokens, token_bytes)) || !elem_aligned(stats, 8) ||
      !elem_aligned(entropy, 4) || !elem_aligned(grad_logp, 4) || !elem_aligned(grad_entropy, 4) ||
      !elem_aligned(dlogits, es))
    return DYT_ERR_INVALID_VALUE;
  const float C = (float)(dyt::loss::kLog2eD / temperature);
  if (!(C > 0.0f) || std::isinf(C)) return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  const LossPlan p = plan_backward(M, N, es, sms);
  LogpGradArgs a = {};
  a.z = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.ignore = ignore_index;
  a.stats = (const float2 *)stats;
  a.entropy = entropy;
  a.da = grad_logp;
  a.db = grad_entropy;
  a.dz = dlogits;
  a.lddz = lddl;
  a.M = M;
  a.N = N;
  a.S = p.S;
  a.wide_tokens = token_bytes == 8;
  a.lines = whole_lines(logits, ld, dlogits, lddl, es);
  a.C = C;
  a.inv_t = 1.0 / temperature;
  const bool shift = !same_offset(logits, dlogits) || !vec_pitch(ld - lddl, es);
  return with_type(dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    PdlConfig lc((unsigned)p.grid, p.block, 0, (cudaStream_t)stream);
    const auto k = dyt::loss::grad_kernel<T, dyt::loss::LogpGradRow>(p.cta, shift);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, k, a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpLogpBackward, &p, (int)(16 / sizeof(T)), 1, 0);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);
}

}  // extern "C"
