// Host planning that the norms share: how a row is spread over lanes, and the
// walk of a launch over the rows (see dyt_norm.cuh).
#pragma once

#include <algorithm>
#include <cstdint>

#include "dyt_host.h"
#include "dyt_norm.cuh"

namespace dyt {
namespace norm {
namespace host {

using namespace dyt::host;

// How a row is spread over lanes.
struct RowPlan {
  int V = 1, L = 1, NV = 0;
  int block = 0;         // threads of a CTA
  int rows = 1;          // rows side by side in a CTA
  bool group = false;    // a row takes several warps
  bool ragged = false;   // rows off 16-byte boundaries, or of no whole vectors
  bool rowlong = false;  // too long for a CTA's registers
  int cluster = 0;       // CTAs that share a row in their registers
  int cols = 0;          // columns of each
};

inline int pow2_at_least(int64_t v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// vec: elements of 16 bytes. aligned: every row of every tensor is whole aligned vectors. E: elements a lane holds.
inline RowPlan plan_rows(int64_t M, int64_t N, int vec, bool aligned, int E, int sms) {
  RowPlan p;
  const int64_t lanes = aligned ? ceil_div(N / vec, E / vec) : ceil_div(N, E);
  p.ragged = !aligned;
  if (lanes > kBlock) {
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
  // Ragged rows keep two slots more per row: half the threads where that is up to as many as its lanes fill.
  int block = p.ragged && p.L < 8 ? kBlock / 2 : kBlock;
  // Few short rows: smaller CTAs, so that more SMs take part.
  while (!p.group && block > 128 && ceil_div(M, block / p.L) < sms) block >>= 1;
  p.rows = block / p.L;
  p.block = p.rows * p.L;
  return p;
}

// The walk of `grid` CTAs over the rows of tensors with pitches lds (the inputs, then the output).
inline Walk walk_of(const RowPlan &p, int64_t M, int64_t N, int64_t grid, const int64_t *lds, int n, size_t elem,
                        int plane_slots) {
  Walk w = {};
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

inline bool param_ok(const void *p, int dt) { return p == nullptr || elem_aligned(p, dsize(dt)); }

}  // namespace host
}  // namespace norm
}  // namespace dyt
