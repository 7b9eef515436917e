// Policy loss entry points (declared in include/dyt.h): argument checks, launch
// plans and dispatch of the kernels in dyt_loss.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dyt.h"
#include "dyt_host.h"
#include "dyt_loss.cuh"

namespace {

using namespace dyt::host;
using dyt::loss::LossArgs;
using dyt::loss::LossGradArgs;

constexpr int kOpLossForward = 7, kOpLossBackward = 8;  // dyt_launch_info::op
// The forward: 512 threads on an SM, their rings full of shared memory.
constexpr int kRowsPerSm = 512;
constexpr int kMostParts = 256;  // parts of a row, at most
constexpr int kFinishCtasPerSm = 2;

constexpr int kGradBlock = 256;
// CTAs that an SM holds (the kernel's launch bounds). Few rows are split into as many parts as there is room
// for at once: 64 x 131072 bf16 6.2 us, in 1.6 times as many parts 7.7; 300 x 50001 11.7 and 13.2.
constexpr int kGradCtasPerSm = dyt::loss::kGradCtas;
// Rows of at most kWarpRow bytes take a warp, unless there are fewer of them than kCtaRowsPerSm an SM
// (1000 x 2000 bf16, a CTA each, 4.0 us, a warp each 4.3).
constexpr int64_t kWarpRow = 8192;
constexpr int kCtaRowsPerSm = 8;
constexpr int64_t kGradPart = 65536;  // the largest part of a row, bytes
constexpr int64_t kGradPartMin = 4096;  // and the smallest

template <typename F>
dyt_status with_type(int xd, F &&f) {
  switch (xd) {
    case DYT_F32: return f(float{});
    case DYT_BF16: return f(__nv_bfloat16{});
    case DYT_F16: return f(__half{});
  }
  return DYT_ERR_UNSUPPORTED_DTYPE;
}

// Parts of a row and CTAs.
struct LossPlan {
  bool cta;      // backward: a part of a row is a CTA's, else a warp's
  int S;         // parts of a row
  int most;      // forward: the parts that there is room for
  int block;
  int64_t grid;  // CTAs
  int finish;    // forward: CTAs of the second kernel
  size_t off_sums, off_done, bytes;  // forward: the workspace
};

LossPlan plan_forward(int64_t M, int64_t N, size_t es, int sms) {
  LossPlan p = {};
  const int64_t bytes = N * (int64_t)es, warps = (int64_t)sms * (kRowsPerSm / 32);
  const int64_t batches = std::max<int64_t>(1, ceil_div(bytes, 16) / (dyt::loss::kBatch * 32));
  p.S = dyt::loss::choose_parts((float)M, (float)warps, (int)std::min<int64_t>(batches, kMostParts),
                                (int)std::min<int64_t>(batches, INT32_MAX));
  p.most = (int)std::max<int64_t>(p.S, std::min<int64_t>(batches, dyt::loss::kListedParts));
  const int64_t items = M * p.S;
  // few items: small CTAs, one warp's work after the other over all SMs
  p.block = dyt::loss::kRowsBlock;
  while (p.block > 32 && ceil_div(items, p.block / 32) < 2 * (int64_t)sms) p.block >>= 1;
  p.grid = std::min<int64_t>(ceil_div(items, p.block / 32), (int64_t)sms * (kRowsPerSm / p.block));
  const int64_t per = p.most > dyt::loss::kThreadParts ? dyt::loss::kFinishBlock / 32 : dyt::loss::kFinishBlock;
  p.finish = (int)std::min<int64_t>(ceil_div(M, per), (int64_t)sms * kFinishCtasPerSm);
  p.off_sums = ((size_t)M * (size_t)p.most * sizeof(float2) + 15) & ~(size_t)15;
  p.off_done = p.off_sums + (size_t)p.finish * sizeof(double);
  p.bytes = (p.off_done + 2 * sizeof(unsigned) + 15) & ~(size_t)15;
  return p;
}

// Few rows are split until every SM has its CTAs, long ones into parts of kGradPart bytes.
LossPlan plan_backward(int64_t M, int64_t N, size_t es, int sms) {
  LossPlan p = {};
  const int64_t bytes = N * (int64_t)es;
  const int64_t slots = (int64_t)sms * kGradCtasPerSm;
  p.cta = bytes > kWarpRow || M < (int64_t)sms * kCtaRowsPerSm;
  p.S = 1;
  p.block = kGradBlock;
  if (p.cta)
    p.S = (int)std::max<int64_t>(M < slots ? std::max<int64_t>(1, std::min(slots / M, bytes / kGradPartMin)) : 1,
                                 ceil_div(bytes, kGradPart));
  const int64_t items = p.cta ? M * p.S : ceil_div(M, kGradBlock / 32);
  p.grid = std::min<int64_t>(items, (int64_t)1 << 30);
  return p;
}

void record(int op, const LossPlan *p, int vec, int kernels, size_t ws) {
  dyt_launch_info i = {};
  i.op = op;
  i.kernels = kernels;
  i.workspace_bytes = (int64_t)ws;
  if (p) {
    i.path = p->cta ? 2 : 1;
    i.vec = vec;
    i.block = p->block;
    i.grid = (int)p->grid;
    i.row_lanes = i.rows_per_step = p->cta ? 1 : p->block / 32;
    i.col_chunks = p->S;
    i.pack_rows = 1;
  }
  record_info(i);
}

bool finite_positive(double v) { return v > 0.0 && std::isfinite(v); }

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
  // A list for few rows only: every CTA reads all the weights, and a warp looks
  // up at most 32 items in it. Small CTAs have little work to spread.
  a.listed = weight != nullptr && M <= dyt::loss::kMaxListed && p.block == dyt::loss::kRowsBlock &&
             M * p.most <= 32 * p.grid * (p.block / 32);
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
  // Neighbouring vectors of a ragged row share lines, so evicting a line after
  // its first read costs 4% there (4096 x 32003 fp16 82.3 and 78.8 us); on whole
  // lines it gains 1% (8192 x 131072 bf16 632 and 628).
  a.lines = (((uintptr_t)logits | (uintptr_t)dlogits | (uintptr_t)((uint64_t)ld * es) | (uintptr_t)((uint64_t)lddl * es)) &
             127u) == 0;
  const bool shift = !same_offset(logits, dlogits) || !vec_pitch(ld - lddl, es);
  return with_type(dtype, [&](auto t) -> dyt_status {
    using T = decltype(t);
    PdlConfig lc((unsigned)p.grid, p.block, 0, (cudaStream_t)stream);
    const auto k = p.cta ? (shift ? dyt::loss::loss_grad_kernel<T, true, true> : dyt::loss::loss_grad_kernel<T, true, false>)
                         : (shift ? dyt::loss::loss_grad_kernel<T, false, true> : dyt::loss::loss_grad_kernel<T, false, false>);
    const cudaError_t e = cudaLaunchKernelEx(&lc.cfg, k, a);
    if (e != cudaSuccess) return cuda_fail(e);
    record(kOpLossBackward, &p, (int)(16 / sizeof(T)), 1, 0);
    return DYT_OK;
  });
} catch (...) {
  return cuda_fail(cudaErrorMemoryAllocation);
}

}  // extern "C"
