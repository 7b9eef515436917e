// Policy loss entry points (declared in include/dyt.h): argument checks, launch
// plans and dispatch of the kernels in dyt_loss.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dyt.h"
#include "dyt_host.h"
#include "dyt_loss.cuh"
#include "dyt_loss_plan.h"

namespace {

using namespace dyt::host;
using namespace dyt::loss::host;
using dyt::loss::LossArgs;
using dyt::loss::LossGradArgs;

constexpr int kOpLossForward = 7, kOpLossBackward = 8;  // dyt_launch_info::op

}  // namespace

extern "C" {

size_t dyt_policy_loss_workspace_bytes(int64_t M, int64_t N, dyt_dtype dtype) try {
  if (check_shape(M, N, dtype) != DYT_OK || M == 0 || N == 0) return 0;
  int dev = 0, sms = 0;
  if (current_sms(&dev, &sms) != DYT_OK) return 0;
  return plan_forward(M, N, dsize(dtype), sms).bytes;
} catch (...) {
  return 0;
}

dyt_status dyt_policy_loss_forward(const void *logits, int64_t ld, const void *tokens, int token_bytes,
                                   const float *old_logp, const float *ref_logp, const float *advantage,
                                   const float *weight, double clip_low, double clip_high, double kl_coef,
                                   double temperature, float *loss, float *logp, float *stats, float *coef, int64_t M,
                                   int64_t N, dyt_dtype dtype, void *workspace, size_t workspace_bytes,
                                   dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, dtype);
  if (st != DYT_OK) return st;
  if (check_pitch(M, N, ld) != DYT_OK || (token_bytes != 4 && token_bytes != 8)) return DYT_ERR_INVALID_VALUE;
  if (!(clip_low >= 0.0) || !std::isfinite(clip_low) || !(clip_high >= 0.0) || !std::isfinite(clip_high) ||
      !std::isfinite(kl_coef) || !finite_positive(temperature))
    return DYT_ERR_INVALID_VALUE;
  if (!loss || !elem_aligned(loss, 4) || (M > 0 && N == 0)) return DYT_ERR_INVALID_VALUE;
  const cudaStream_t s = (cudaStream_t)stream;
  if (M == 0) {
    const cudaError_t e = cudaMemsetAsync(loss, 0, sizeof(float), s);  // the empty sum
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpLossForward, nullptr, 0, 0, 0);
    return DYT_OK;
  }
  if (M == 1) ld = N;  // one row has no pitch
  const size_t es = dsize(dtype);
  if (!logits || !tokens || !old_logp || !advantage || !logp || !stats || !coef || !workspace ||
      !elem_aligned(logits, es) || !elem_aligned(tokens, token_bytes) || !elem_aligned(old_logp, 4) ||
      !elem_aligned(ref_logp, 4) || !elem_aligned(advantage, 4) || !elem_aligned(weight, 4) ||
      !elem_aligned(logp, 4) || !elem_aligned(stats, 8) || !elem_aligned(coef, 4) || !aligned16(workspace))
    return DYT_ERR_INVALID_VALUE;
  const float C = (float)(dyt::loss::kLog2eD / temperature);
  if (!(C > 0.0f) || std::isinf(C)) return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  const LossPlan p = plan_forward(M, N, es, sms);
  if (workspace_bytes < p.bytes) return DYT_ERR_WORKSPACE_TOO_SMALL;
  LossArgs a = {};
  a.z = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.advantage = advantage;
  a.weight = weight;
  a.loss = loss;
  a.logp = logp;
  a.stats = (float2 *)stats;
  a.coef = coef;
  a.parts = (float2 *)workspace;
  a.sums = (double *)((char *)workspace + p.off_sums);
  a.done = (unsigned *)((char *)workspace + p.off_done);
  a.M = M;
  a.N = N;
  a.S = p.S;
  a.most = p.most;
  a.batches = (int)ceil_div(ceil_div(N * (int64_t)es, 16), dyt::loss::kBatch * 32);
  a.listed = weight != nullptr && lists_rows(p, M);
  a.aligned = N % (16 / (int64_t)es) == 0 && aligned16(logits) && vec_pitch(ld, es);
  a.wide_tokens = token_bytes == 8;
  a.C = C;
  a.inv_t = 1.0 / temperature;
  a.lo = 1.0 - clip_low;
  a.hi = 1.0 + clip_high;
  a.kl = kl_coef;
  return with_type(dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    const size_t smem = dyt::loss::rows_smem(p.block);
    const dyt_status ready = prepare_smem(dev, (const void *)dyt::loss::loss_rows_kernel<T>, (int)smem);
    if (ready != DYT_OK) return ready;
    PdlConfig lc((unsigned)p.grid, p.block, smem, s);
    cudaError_t e = cudaLaunchKernelEx(&lc.cfg, dyt::loss::loss_rows_kernel<T>, a);
    if (e != cudaSuccess) return cuda_fail(e);
    PdlConfig lf((unsigned)p.finish, dyt::loss::kFinishBlock, 0, s);
    e = cudaLaunchKernelEx(&lf.cfg, dyt::loss::loss_finish_kernel<T>, a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpLossForward, &p, (int)(16 / sizeof(T)), 2, p.bytes);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);  // the host ran out of memory for the per-device facts
}

dyt_status dyt_policy_loss_backward(const void *logits, int64_t ld, const void *tokens, int token_bytes,
                                    const float *stats, const float *coef, const float *grad, double temperature,
                                    void *dlogits, int64_t lddl, int64_t M, int64_t N, dyt_dtype dtype,
                                    dyt_stream_t stream) try {
  dyt_status st = check_shape(M, N, dtype);
  if (st != DYT_OK) return st;
  if (check_pitch(M, N, ld) != DYT_OK || check_pitch(M, N, lddl) != DYT_OK || (token_bytes != 4 && token_bytes != 8) ||
      !finite_positive(temperature))
    return DYT_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) {
    record(kOpLossBackward, nullptr, 0, 0, 0);
    return DYT_OK;
  }
  if (M == 1) ld = lddl = N;  // one row has no pitch
  const size_t es = dsize(dtype);
  if (!logits || !tokens || !stats || !coef || !dlogits || !elem_aligned(logits, es) ||
      !elem_aligned(tokens, token_bytes) || !elem_aligned(stats, 8) || !elem_aligned(coef, 4) ||
      !elem_aligned(grad, 4) || !elem_aligned(dlogits, es))
    return DYT_ERR_INVALID_VALUE;
  const float C = (float)(dyt::loss::kLog2eD / temperature);
  if (!(C > 0.0f) || std::isinf(C)) return DYT_ERR_INVALID_VALUE;
  int dev = 0, sms = 0;
  st = current_sms(&dev, &sms);
  if (st != DYT_OK) return st;
  const LossPlan p = plan_backward(M, N, es, sms);
  LossGradArgs a = {};
  a.z = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.stats = (const float2 *)stats;
  a.coef = coef;
  a.grad = grad;
  a.dz = dlogits;
  a.lddz = lddl;
  a.M = M;
  a.N = N;
  a.S = p.S;
  a.wide_tokens = token_bytes == 8;
  a.C = C;
  a.inv_t = 1.0 / temperature;
  a.lines = whole_lines(logits, ld, dlogits, lddl, es);
  const bool shift = !same_offset(logits, dlogits) || !vec_pitch(ld - lddl, es);
  return with_type(dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    PdlConfig lc((unsigned)p.grid, p.block, 0, (cudaStream_t)stream);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, dyt::loss::grad_kernel<T, dyt::loss::LossGradRow>(p.cta, shift), a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpLossBackward, &p, (int)(16 / sizeof(T)), 1, 0);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);
}

}  // extern "C"
