// Host planning that the passes over logits share: parts of a row, CTAs and
// workspaces (see dyt_loss.cuh).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dyt_host.h"
#include "dyt_loss.cuh"

namespace dyt {
namespace loss {
namespace host {

using namespace dyt::host;

// The forward: 512 threads on an SM, their rings full of shared memory.
constexpr int kRowsPerSm = 512;
constexpr int kMostParts = 256;  // parts of a row, at most
constexpr int kFinishCtasPerSm = 2;

constexpr int kGradBlock = 256;
// CTAs that an SM holds (the kernel's launch bounds). Few rows are split into as many parts as there is room
// for at once: 64 x 131072 bf16 6.2 us, in 1.6 times as many parts 7.7; 300 x 50001 11.7 and 13.2.
constexpr int kGradCtasPerSm = kGradCtas;
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

inline LossPlan plan_forward(int64_t M, int64_t N, size_t es, int sms) {
  LossPlan p = {};
  const int64_t bytes = N * (int64_t)es, warps = (int64_t)sms * (kRowsPerSm / 32);
  const int64_t batches = std::max<int64_t>(1, ceil_div(bytes, 16) / (kBatch * 32));
  p.S = choose_parts((float)M, (float)warps, (int)std::min<int64_t>(batches, kMostParts),
                                (int)std::min<int64_t>(batches, INT32_MAX));
  p.most = (int)std::max<int64_t>(p.S, std::min<int64_t>(batches, kListedParts));
  const int64_t items = M * p.S;
  // few items: small CTAs, one warp's work after the other over all SMs
  p.block = kRowsBlock;
  while (p.block > 32 && ceil_div(items, p.block / 32) < 2 * (int64_t)sms) p.block >>= 1;
  p.grid = std::min<int64_t>(ceil_div(items, p.block / 32), (int64_t)sms * (kRowsPerSm / p.block));
  const int64_t per = p.most > kThreadParts ? kFinishBlock / 32 : kFinishBlock;
  p.finish = (int)std::min<int64_t>(ceil_div(M, per), (int64_t)sms * kFinishCtasPerSm);
  p.off_sums = ((size_t)M * (size_t)p.most * sizeof(float2) + 15) & ~(size_t)15;
  p.off_done = p.off_sums + (size_t)p.finish * sizeof(double);
  p.bytes = (p.off_done + 2 * sizeof(unsigned) + 15) & ~(size_t)15;
  return p;
}

// Few rows are split until every SM has its CTAs, long ones into parts of kGradPart bytes.
inline LossPlan plan_backward(int64_t M, int64_t N, size_t es, int sms) {
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

inline void record(int op, const LossPlan *p, int vec, int kernels, size_t ws) {
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

inline bool finite_positive(double v) { return v > 0.0 && std::isfinite(v); }

// Whether the forward's first kernel lists the rows that count. A list for few rows only: every CTA
// reads all the weights, and a warp looks up at most 32 items in it. Small CTAs have little work to spread.
inline bool lists_rows(const LossPlan &p, int64_t M) {
  return M <= kMaxListed && p.block == kRowsBlock && M * p.most <= 32 * p.grid * (p.block / 32);
}

// Whether every row of the backward is whole 128-byte lines. Neighbouring vectors of a ragged row share
// lines, so evicting a line after its first read costs 4% there (4096 x 32003 fp16 82.3 and 78.8 us); on
// whole lines it gains 1% (8192 x 131072 bf16 632 and 628).
inline bool whole_lines(const void *z, int64_t ld, const void *dz, int64_t lddz, size_t es) {
  return (((uintptr_t)z | (uintptr_t)dz | (uintptr_t)((uint64_t)ld * es) | (uintptr_t)((uint64_t)lddz * es)) & 127u) == 0;
}

}  // namespace host
}  // namespace loss
}  // namespace dyt
