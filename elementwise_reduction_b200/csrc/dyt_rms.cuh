// Root-mean-square norm with the residual's addition, forward (also with an 8-bit
// output and its scales) and backward, for sm_100a over the rows of an M x N matrix.
//
//   h_j  = x_j + residual_j   (binary32; stored rounded; x_j without a residual)
//   rstd = (sum_j h_j^2 / N + eps)^-1/2,   y_j = gamma_j h_j rstd
//   scale = max(max_j |y_j|, 2^-100) / 448 over the row, or over 128 columns;  q_j = e4m3(y_j / scale)
//   n_j  = h_j rstd,  g_j = gamma_j dy_j,  c = sum_j g_j n_j / N
//   dx_j = rstd (g_j - n_j c) + dh_j,   dgamma_j = sum_i dy_ij n_ij
//
// Bound by memory, as layer norm is, and mostly laid out as it: a row is read once
// into the ring of RowFeed and kept in registers between its sum and its outputs,
// the same columns of every row in the same lane. The norm is of the sum before it
// is rounded to the stored residual stream, so y has one rounding. The 8-bit output
// is of the same y, by the quotient that its definition names; where one scale is the
// whole row's, the largest |y| takes an exchange of its own behind the sum's.
#pragma once

#include <cfloat>
#include <type_traits>

#include "dyt_cluster.cuh"
#include "dyt_norm.cuh"
#include "dyt_steal.cuh"

namespace dyt {
namespace norm {

struct RmsArgs {
  const void *x;
  int64_t ldx;
  const void *res;    // with a residual
  int64_t ldr;
  const void *gamma;  // NULL: 1
  void *y;            // T, or e4m3
  int64_t ldy;
  void *h;            // with a residual
  int64_t ldh;
  float *rstd;        // NULL: not written
  float *scale;       // [M] or [M][groups]
  int gamma_dt;
  float eps;
  int groups;         // scales a row: 1, or one for each kScaleCols columns (grouped)
  int grouped;
  int steal;          // a CTA an item, and work is taken from those that do not run yet; else a fixed share
  int64_t items;      // a CTA's rows of a step each
  int cols;           // clusters: columns of a CTA, a multiple of kScaleCols
  Walk w;             // (a step is 0: rows come in no order)
};

struct RmsGradArgs {
  const void *h;
  int64_t ldh;
  const void *dy;
  int64_t lddy;
  const void *dres;   // the gradient of the stored sum (with one)
  int64_t lddr;
  const void *gamma;  // NULL: 1
  const float *rstd;
  void *dx;
  int64_t lddx;
  double *parts;      // [CTA][N] column sums; NULL: the one CTA's are dgamma
  void *dgamma;       // then (NULL: not wanted)
  int gamma_dt;
  int64_t inc_dx;
  int cols;           // clusters: columns of a CTA
  Walk w;             // inc[0 .. 2]: of h, dy and dres
};

constexpr int kScaleCols = 128;
constexpr int kClusterMost = 4;  // rows of a cluster side by side, at most
constexpr float kQMax = 448.0f;      // the largest e4m3 value
constexpr float kLeastTop = 0x1p-100f;  // a row of zeros has a scale all the same: nothing is divided by 0

__device__ __forceinline__ float lanes_max(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// A CTA's place among those that share its rows (one, but for kCluster): its number of them and its stretch's first
// column; `unit` counts the clusters, or the CTAs.
template <int MODE>
struct Share {
  static __device__ __forceinline__ uint32_t rank() { return in_cluster(MODE) ? cluster_rank() : 0; }
  static __device__ __forceinline__ uint32_t ctas() { return in_cluster(MODE) ? cluster_ctas() : 1; }
  static __device__ __forceinline__ uint32_t unit() { return blockIdx.x / ctas(); }
  static __device__ __forceinline__ uint32_t units() { return gridDim.x / ctas(); }
  static __device__ __forceinline__ int first(int cols) { return in_cluster(MODE) ? (int)cluster_rank() * cols : 0; }
};
// The walk over a CTA's stretch of the rows' columns.
template <int MODE>
using ShareWalk = std::conditional_t<in_cluster(MODE), Walk, const Walk &>;
__device__ __forceinline__ void cut(Walk &w, int first, int cols, int V) {  // V: elements of a vector
  const int left = (int)w.N - first;
  w.N = left < cols ? left : cols;
  w.NV = (int)w.N / V;
}
__device__ __forceinline__ const void *param_from(const void *p, int dt, int first) {
  return p ? static_cast<const char *>(p) + (int64_t)first * (dt == DYT_F32 ? 4 : 2) : p;
}

// A group's scale from its largest |y|, and the quotients by it.
struct Scale {
  float s, inv, rest;  // the scale, its inverse from below, and what that lacks (both 0 for an infinite scale)
  __device__ __forceinline__ explicit Scale(float top) {
    s = max_nan(top, kLeastTop) * (1.0f / kQMax);
    inv = rcp_approx(s) * (1.0f - 0x1p-22f);
    rest = fmaf(-inv, fminf(s, FLT_MAX), 1.0f) * inv;  // (not negative: no sum of it turns a -0)
  }
  // The binary32 nearest to y / s (but for quotients within 2^-20 units of the middle of two, and scales over 2^100,
  // whose rest is subnormal): 1 / s in two parts, 45 bits of it. By one rounded part a value in four is a unit in the
  // last place off, and one e4m3 value in 50000 lies on the other side of a tie.
  __device__ __forceinline__ float2 quotient(float2 y) const { return fma2(y, f2(inv), mul2(y, f2(rest))); }
};

// Two values rounded to e4m3 (nearest even, at most 448; NaN stays): a in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float2 v) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
  return r;
}

// V values as e4m3 bytes at p (V bytes apart from a V-byte boundary).
template <int V>
__device__ __forceinline__ void store_e4m3(unsigned char *p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = (unsigned char)e4m3_pair(make_float2(f[0], 0.0f));
  } else {
    uint32_t w[(V + 3) / 4];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const uint32_t b = e4m3_pair(make_float2(f[i], f[i + 1]));
      if (i % 4) w[i / 4] |= b << 16;
      else w[i / 4] = b;
    }
    if constexpr (V == 2) *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
    else if constexpr (V == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  }
}

// A lane's outputs as e4m3 bytes to the row at `out`, where the row is (`in`). RAGGED: they pass through `room`, the
// slots that the row came from, where they lie as in their 16-byte chunks of memory. (Single bytes instead, 32 a store,
// when both were there: 8191 x 1001 fp16 10.2 us, so 9.9; with a residual 100003 x 700 bf16 133 and 125, 4096 x 20481
// 254 and 227; but 100003 x 100 31.7 and 34.2. All widths go this way: a second way for the narrow ones is not built.)
template <typename T, int E, bool RAGGED, int MODE, typename Feed>
__device__ __forceinline__ void store_bytes(unsigned char *out, const float2 (&f)[E / 2], const Place<MODE> &p,
                                            const Feed &feed, int NV, unsigned char *room, bool in) {
  constexpr int V = 16 / (int)sizeof(T);
  if constexpr (!RAGGED) {
    if (!in) return;
#pragma unroll
    for (int k = 0; k < E / V; ++k)
      if (p.lane + k * p.L < NV)
        store_e4m3<V>(out + (p.lane + k * p.L) * V, *reinterpret_cast<const float(*)[V]>(f + k * (V / 2)));
  } else {
    unsigned char *o = out + column<V, E, true, MODE>(p.L, p.lane - p.at, 0);  // the warp's stretch
    const int len = in ? feed.need / (int)sizeof(T) : 0, d = (int)((uintptr_t)o & 15u), end = d + len;
    unsigned char *s = room + d + p.at;
    __syncwarp();  // all lanes have what they read there
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint32_t b = e4m3_pair(f[i / 2]);
      s[i * p.seg()] = (unsigned char)b;
      s[(i + 1) * p.seg()] = (unsigned char)(b >> 8);
    }
    __syncwarp();
    if (len > 0) {
#pragma unroll
      for (int k = 0; k <= E / 16; ++k) {
        const int c = (p.at + k * p.seg()) * 16;
        if (c >= d && c + 16 <= end) *reinterpret_cast<uint4 *>(o - d + c) = *reinterpret_cast<const uint4 *>(room + c);
      }
      // the bytes of chunks that are not all the stretch's, at its two ends
      const int tail = end & ~15;
      if (d)
        for (int c = d + p.at; c < 16 && c < end; c += p.seg()) o[c - d] = room[c];
      if (tail >= d)
        for (int c = tail + p.at; c < end; c += p.seg()) o[c - d] = room[c];
    }
  }
}

// Scales of kScaleCols columns each. A lane's elements fall into slabs that lie in one group: its
// vectors (aligned rows), or four elements (ragged ones, seg <= 32 apart). The slab's lanes are
// reduced by a butterfly; rows in less than a warp may have several slabs of one group.
template <typename T, int E, bool RAGGED, int MODE>
struct Slabs {
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int W = RAGGED ? 4 : V;  // elements of a slab
  static constexpr int n = E / W;
  static __device__ __forceinline__ int lanes(const Place<MODE> &p) {
    return RAGGED || p.seg() < kScaleCols / V ? p.seg() : kScaleCols / V;
  }
  // The group of slab s.
  static __device__ __forceinline__ int group(const Place<MODE> &p, int s) {
    return column<V, E, RAGGED, MODE>(p.L, p.lane, s * W) / kScaleCols;
  }
  // top[s]: the largest of the lane's slab s; becomes that of the slab's group.
  static __device__ __forceinline__ void join(float (&top)[n], const Place<MODE> &p) {
    const int width = lanes(p);
#pragma unroll
    for (int s = 0; s < n; ++s) top[s] = lanes_max(top[s], width);
    if constexpr (shares_warp(MODE)) {  // (a slab's group is the same for all its lanes)
      float all[n];
#pragma unroll
      for (int s = 0; s < n; ++s) {
        all[s] = top[s];
#pragma unroll
        for (int o = 0; o < n; ++o)
          if (o != s && group(p, o) == group(p, s)) all[s] = max_nan(all[s], top[o]);
      }
#pragma unroll
      for (int s = 0; s < n; ++s) top[s] = all[s];
    }
  }
};

// ---- forward: a row in registers -------------------------------------------------

constexpr int kRmsFwdStages = 3;
// Elements of a row a lane holds in rows of at most 32 times as many: with 32 of them and the lanes' number unknown
// ragged 16-bit rows spill (100003 x 255 bf16 with a residual 92 us, with 16 49).
constexpr int kNarrowElems = 16;
constexpr int kNarrowBlock = 128;  // threads of a CTA of rows in a warp or less
template <typename T, int E>
__host__ __device__ constexpr size_t rms_fwd_smem(int block, int L, bool ragged, bool res) {
  return (size_t)kRmsFwdStages * (res ? 2 : 1) * row_slots<T, E>(block, L, ragged) * 16;
}

// What a CTA leaves whose wait for an answer ran out of its limit, which the hardware does not let happen: the row
// that the answer named is not done, and the CTA's first row says so with NaN.
template <typename T, bool Q>
__device__ __noinline__ void give_up(const RmsArgs &a, int64_t row) {
  const float nan = __int_as_float(0x7FC00000);
  if (a.rstd) a.rstd[row] = nan;
  if constexpr (Q) a.scale[row * a.groups] = nan;
  else static_cast<T *>(a.y)[row * a.ldy] = from_f32<T>(nan);
}

// RES: with a residual. Q: 8-bit output with scales. A CTA has a row of several warps, or a few smaller ones side by
// side; several CTAs share an SM, and those that run take the rows of those that were not launched yet
// (dyt_steal.cuh): an SM gets as many rows as it has time for. With MODE kCluster the row's warps are in several CTAs
// (dyt_cluster.cuh), and a cluster has a fixed share of the rows.
// Measured with a residual, bf16: 16384 x 4096 80.5 us (6.65 TB/s), 65536 x 1024 80.2 (6.7), 4096 x 20480 by clusters
// of 2 117 (5.7); without one, 100003 x 255 binary32 32.4 (6.3). 8-bit, with a residual: 8192 x 8192, a scale for 128
// columns, 72 (6.5); 4096 x 20480 103 with a scale for 128 columns, and 103 with one a row (with its largest value in
// the sum's exchange, from gamma h, 92). Bound by memory; ragged 16-bit rows by instructions, as each element is a load
// from shared memory and a store of its own: 100003 x 255 bf16 44.7 (4.6), 8191 x 1001 fp16 to 8 bits 10.0 (2.5).
template <typename T, int E, int MODE, bool RAGGED, bool RES, bool Q>
__global__ void __launch_bounds__(kBlock, 1) rms_fwd_kernel(const __grid_constant__ RmsArgs a) {
  constexpr bool CLUSTER = in_cluster(MODE), GROUP = in_warps(MODE);
  using Mine = Share<MODE>;
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int P = E / 2;
  constexpr int S = kRmsFwdStages, TN = RES ? 2 : 1;
  using Slab = Slabs<T, E, RAGGED, MODE>;
  __shared__ std::conditional_t<CLUSTER, Meet, float[2][2][kBlock / 32]> red;
  __shared__ Steal queue;
  extern __shared__ __align__(128) unsigned char dyn[];
  pdl_prologue();
  const Place<MODE> p(a.w.L);
  if (dynamic_smem_bytes() < rms_fwd_smem<T, E>((int)blockDim.x, p.L, RAGGED, RES)) return;
  const int col0 = Mine::first(a.cols);
  ShareWalk<MODE> w = a.w;
  if constexpr (CLUSTER) {
    cut(w, col0, a.cols, RAGGED ? 1 : V);
    red.init(p.lane, p.L);
    cluster_sync();
  }
  const bool steal = !CLUSTER && a.steal;
  const int groups = CLUSTER ? ((int)w.N + kScaleCols - 1) / kScaleCols : a.groups;  // of the CTA's stretch
  const int N = (int)w.N;
  const T *src[TN];
  int64_t ld[TN];
  src[0] = static_cast<const T *>(a.x) + col0;
  ld[0] = a.ldx;
  if constexpr (RES) {
    src[1] = static_cast<const T *>(a.res) + col0;
    ld[1] = a.ldr;
  }
  // Item i: rows i rows .. i rows + rows - 1. (M for the row of none.) With fixed shares the CTA's items lie a grid
  // apart.
  const int64_t M = w.M;
  auto row_of = [&](int64_t item) {
    const int64_t r = GROUP ? item : item * w.rows + p.mine;
    return item >= 0 && r < M ? r : M;
  };
  int64_t item = Mine::unit(), next = -1;  // this one and the one after, -1: none
  uint32_t asked = 0;                    // answers taken
  RowFeed<T, E, TN, S, RAGGED, MODE> feed(dyn, src, ld, p, w, row_of(item));
  static_assert(S == 3, "this row and the next one are on their way");
  auto fetch = [&](int64_t i) {
    const int64_t r = row_of(i);
    feed.seek(src, ld, p, r);
    feed.issue(p, w, r < M, r);
  };
  fetch(item);
  if (steal) {
    if (threadIdx.x == 0) queue.init();
    __syncthreads();
    if (threadIdx.x == 0) queue.ask();
  }
  float2 gam[P];
  load_pairs<V, E, RAGGED, MODE>(param_from(a.gamma, a.gamma_dt, col0), a.gamma_dt, p, N, 1.0f, gam);
  const float inv_n = w.inv_n;
  const int warps = GROUP ? p.L / 32 : 1, wl = (int)threadIdx.x & 31;
  bool lost = false;
  // CLUSTER: what each of the row's warps has, two for a lane of every warp; NaN once something did not come. step: 0,
  // 1, 2, ...
  auto meet = [&](int step, float v) {
    const float nan = __int_as_float(0x7FC00000);
    if constexpr (CLUSTER) {
      red.put(step, lost ? nan : v, p.lane, p.L);
      if (!lost) lost = !red.wait(step, p.lane, p.L);
      if (!lost) return make_float2(red.of[step & 1][wl], red.of[step & 1][wl + 32]);
    }
    return make_float2(nan, nan);
  };
  auto take = [&](int64_t last) {
    if (steal) return queue.take(asked++ & 1u);
    return last + Mine::units() < a.items ? last + Mine::units() : (int64_t)-1;
  };
  // All have taken the answer, which was `got`: the next question. (Groups meet here in any case.)
  auto taken = [&](int64_t &got) {
    if (!steal) {
      if constexpr (MODE == kGroup) __syncthreads();
      return;
    }
    if (__syncthreads_or(got == Steal::kLost)) {  // (whichever thread it was: all stop asking)
      lost = true;
      got = -1;
    }
    if (got >= 0 && threadIdx.x == 0) queue.ask();
  };
  next = take(item);
  taken(next);
  fetch(next);
#pragma unroll 1
  for (int it = 0; item >= 0; ++it) {
    const int64_t row = row_of(item);
    const bool in = GROUP || row < M;  // (lanes without a row take all steps with the others)
    feed.wait();
    float2 v[P];
    feed.read(0, src[0], ld[0], row, p, w, v);
    if constexpr (RES) {
      float2 r[P];
      feed.read(1, src[1], ld[1], row, p, w, r);
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = add2(v[i], r[i]);
    }
    unsigned char *const room = feed.mine + feed.rd;  // the row's slots, free until the row after next is copied
    feed.advance(w);
    int64_t after = -1;
    if (next >= 0) after = take(next);
    fetch(after);
    float2 t[2] = {f2(0.0f), f2(0.0f)};  // what lies past the row's end is zero
#pragma unroll
    for (int i = 0; i < P; ++i) t[i & 1] = fma2(v[i], v[i], t[i & 1]);
    t[0] = add2(t[0], t[1]);
    float q = t[0].x + t[0].y;
    if (RES && in) store_pairs<T, E, RAGGED>(static_cast<T *>(a.h) + row * a.ldh + col0, v, p, feed, w.NV, N);
    q = GROUP ? warp_sum(q) : lanes_sum(q, p.L);
    const int par = it & 1;
    if constexpr (CLUSTER) {
      const float2 o = meet(Q && !a.grouped ? 2 * it : it, q);
      q = warp_sum(o.x + o.y);
    } else if constexpr (GROUP) {
      if (wl == 0) red[par][0][p.lane / 32] = q;
      taken(after);
      // up to 16 warps, one a lane of each half
      q = lanes_sum((wl & 15) < warps ? red[par][0][wl & 15] : 0.0f, 16);
    } else {
      taken(after);
    }
    const float rstd = rsqrtf(fmaf(q, inv_n, a.eps));
    if (a.rstd && p.lane == 0 && in && Mine::rank() == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(mul2(v[i], f2(rstd)), gam[i]);
    if constexpr (Q) {
      if (a.grouped) {
        float tops[Slab::n];
#pragma unroll
        for (int s = 0; s < Slab::n; ++s) {
          tops[s] = 0.0f;
#pragma unroll
          for (int i = s * Slab::W / 2; i < (s + 1) * Slab::W / 2; ++i)
            tops[s] = max_nan(tops[s], max_nan(fabsf(v[i].x), fabsf(v[i].y)));
        }
        Slab::join(tops, p);
#pragma unroll
        for (int s = 0; s < Slab::n; ++s) {
          const Scale c(tops[s]);
          const int g = Slab::group(p, s);
          // (rows in less than a warp: several slabs may write the same value)
          if (in && g < groups && (p.lane & (Slab::lanes(p) - 1)) == 0)
            a.scale[row * a.groups + col0 / kScaleCols + g] = c.s;
#pragma unroll
          for (int i = s * Slab::W / 2; i < (s + 1) * Slab::W / 2; ++i) v[i] = c.quotient(v[i]);
        }
      } else {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) top = max_nan(top, max_nan(fabsf(v[i].x), fabsf(v[i].y)));
        top = lanes_max(top, p.seg());
        if constexpr (CLUSTER) {
          const float2 o = meet(2 * it + 1, top);
          top = lanes_max(max_nan(o.x, o.y), 32);
        } else if constexpr (GROUP) {
          if (wl == 0) red[par][1][p.lane / 32] = top;
          __syncthreads();
          top = lanes_max((wl & 15) < warps ? red[par][1][wl & 15] : 0.0f, 16);
        }
        const Scale c(top);
        if (p.lane == 0 && in && Mine::rank() == 0) a.scale[row] = c.s;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = c.quotient(v[i]);
      }
      store_bytes<T, E, RAGGED>(static_cast<unsigned char *>(a.y) + row * a.ldy + col0, v, p, feed, w.NV, room, in);
    } else if (in) {
      store_pairs<T, E, RAGGED>(static_cast<T *>(a.y) + row * a.ldy + col0, v, p, feed, w.NV, N);
    }
    item = next;
    next = after;
  }
  cp_async_wait<0>();
  if constexpr (CLUSTER) {
    cluster_sync();  // a CTA ends behind what the others send it
  } else if (lost) {
    __syncthreads();  // behind what the CTA wrote of the row
    if (threadIdx.x == 0) give_up<T, Q>(a, (int64_t)blockIdx.x * (GROUP ? 1 : w.rows));
  }
}

// ---- forward: rows too long for registers ----------------------------------------

// The largest over a CTA (see cta_sum).
__device__ __forceinline__ float cta_max(float v, float *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  v = lanes_max(v, 32);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return lanes_max(lane < warps ? red[lane] : 0.0f, 32);
}

// Rows of more columns than 4 CTAs hold: one CTA reads each row twice (the second time mostly from L2), for its sum of
// squares and for its outputs. A warp takes 32 x C consecutive columns at a time, C = 4 single elements or a vector a
// lane, which are whole groups of kScaleCols. With a scale a row there is a third reading, for the largest value.
// Measured: 512 x 131072 bf16 with a residual 161 us (3.3 TB/s of what one pass would move), to 8 bits with a scale a
// row 232; bound by the wait for the sum, during which the CTA writes nothing.
template <typename T, int V, bool RES, bool Q>
__global__ void __launch_bounds__(1024) rms_fwd_long_kernel(RmsArgs a) {
  constexpr int C = V == 1 ? 4 : V;       // a lane's columns of a step
  constexpr int B = V == 1 ? 4 : 1;       // loads for them
  constexpr int GL = kScaleCols / C;      // lanes of a scale's columns
  using IO = VecIO<T, V>;
  __shared__ float red[2][kMaxWarps];
  pdl_prologue();
  const int64_t N = a.w.N;
  const int lane = threadIdx.x & 31;
  const int64_t c0 = (int64_t)(threadIdx.x >> 5) * (32 * C) + lane * V, step = (int64_t)blockDim.x * C;
  for (int64_t row = blockIdx.x; row < a.w.M; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *r = static_cast<const T *>(a.res) + (RES ? row * a.ldr : 0);
    // the sum at columns c + b 32 V + e, 0 past the end
    auto sum_at = [&](int64_t c, float (&v)[C]) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        float f[V], g[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = 0.0f;
        if (c + b * 32 < N) {
          IO::unpack(load_row<T, V>(x + c + b * 32), f);
          if constexpr (RES) {
            IO::unpack(load_row<T, V>(r + c + b * 32), g);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] += g[e];
          }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) v[b * V + e] = f[e];
      }
    };
    // gamma there; 8 bits: 0 past the end too, where a group's largest value would meet another column's
    auto gamma_at = [&](int64_t c, float (&g)[C]) {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const bool inside = c + b * 32 < N;
        float f[V];
        load_columns<V>(a.gamma, a.gamma_dt, inside ? c + b * 32 : 0, 1.0f, f);
#pragma unroll
        for (int e = 0; e < V; ++e) g[b * V + e] = inside || !Q ? f[e] : 0.0f;
      }
    };
    float s[1] = {0.0f}, top = 0.0f;
#pragma unroll 2
    for (int64_t c = c0; c < N; c += step) {
      float v[C];
      sum_at(c, v);
#pragma unroll
      for (int e = 0; e < C; ++e) s[0] = fmaf(v[e], v[e], s[0]);
    }
    cta_sum(s, red[0]);
    const float rstd = rsqrtf(fmaf(s[0], a.w.inv_n, a.eps));
    if (Q && !a.grouped) {
#pragma unroll 2
      for (int64_t c = c0; c < N; c += step) {
        float v[C], g[C];
        sum_at(c, v);
        gamma_at(c, g);
#pragma unroll
        for (int e = 0; e < C; ++e) top = max_nan(top, fabsf(v[e] * rstd * g[e]));
      }
      top = cta_max(top, red[1]);
    }
    const Scale whole(top);
    if (threadIdx.x == 0) {
      if (a.rstd) a.rstd[row] = rstd;
      if (Q && !a.grouped) a.scale[row] = whole.s;
    }
    // whole warps stay together: a warp's first column decides
    for (int64_t c = c0; c - lane * V < N; c += step) {
      float v[C], g[C];
      sum_at(c, v);
      gamma_at(c, g);
      if constexpr (RES) {
        T *h = static_cast<T *>(a.h) + row * a.ldh + c;
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (c + b * 32 < N) store_row<T, V>(h + b * 32, *reinterpret_cast<const float(*)[V]>(v + b * V));
      }
#pragma unroll
      for (int e = 0; e < C; ++e) v[e] = v[e] * rstd * g[e];
      if constexpr (!Q) {
        T *y = static_cast<T *>(a.y) + row * a.ldy + c;
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (c + b * 32 < N) store_row<T, V>(y + b * 32, *reinterpret_cast<const float(*)[V]>(v + b * V));
      } else {
        unsigned char *y = static_cast<unsigned char *>(a.y) + row * a.ldy + c;
        Scale by = whole;
        if (a.grouped) {
          float t = 0.0f;
#pragma unroll
          for (int e = 0; e < C; ++e) t = max_nan(t, fabsf(v[e]));
          by = Scale(lanes_max(t, GL));
          const int64_t grp = c / kScaleCols;
          if ((lane & (GL - 1)) == 0 && grp < a.groups) a.scale[row * a.groups + grp] = by.s;
        }
#pragma unroll
        for (int e = 0; e < C; e += 2) {
          const float2 q = by.quotient(make_float2(v[e], v[e + 1]));
          v[e] = q.x;
          v[e + 1] = q.y;
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (c + b * 32 < N) store_e4m3<V>(y + b * 32, *reinterpret_cast<const float(*)[V]>(v + b * V));
      }
    }
    __syncthreads();  // (the second exchange of this row is read before the first of the next is written)
  }
}

// ---- backward: a row in registers ------------------------------------------------

template <typename T>
__host__ __device__ constexpr int rms_bwd_stages() {
  return sizeof(T) == 4 ? 2 : 3;
}
template <typename T>
__host__ __device__ constexpr size_t rms_bwd_ring(int block, int L, bool ragged, bool res) {
  return (size_t)rms_bwd_stages<T>() * (res ? 3 : 2) * row_slots<T, kBwdElems>(block, L, ragged) * 16;
}
// Room for `per` elements' column sums of every lane: a copy per group, or per warp of smaller rows.
__host__ __device__ constexpr size_t rms_sums_smem(int block, int L, int per) {
  return (size_t)(block / (L < 32 ? 32 : L)) * per * (L + kSumPad) * sizeof(float);
}
template <typename T>
__host__ __device__ constexpr size_t rms_bwd_smem(int block, int L, bool ragged, bool res) {
  return rms_bwd_ring<T>(block, L, ragged, res) + rms_sums_smem(block, L, 16 / (int)sizeof(T));
}
static_assert(rms_bwd_ring<__half>(32, 32, false, false) >= rms_sums_smem(32, 32, kBwdElems) &&
                  rms_bwd_ring<float>(32, 32, false, false) >= rms_sums_smem(32, 32, kBwdElems),
              "the last column sums take the ring's place");

// flush_columns for one sum a column: a run's sums of the CTA's rows, added in a fixed order and moved to
// the partial sums pg in binary64, or rounded to dgamma (`only`: there are no others).
template <int V, int E, int PER, bool RAGGED, int MODE>
__device__ __forceinline__ void rms_flush(const RmsGradArgs &a, double *pg, const Walk &w, float2 (&dg)[E / 2],
                                          const Place<MODE> &p, bool first, float *sh) {
  const bool only = !in_cluster(MODE) && a.parts == nullptr;
  constexpr bool GROUP = in_warps(MODE);
  const int N = (int)w.N;
  const int copies = !GROUP ? (int)blockDim.x / 32 : w.rows;
  const int copy = !GROUP ? (int)threadIdx.x >> 5 : p.mine;
  const int stride = p.L + kSumPad, plane = PER * stride;
  auto add = [&](int e, int lane, int c) {
    if (c >= N) return;
    const float *q = sh + e * stride + lane;
    double t[2] = {0.0, 0.0};
    for (int w = 0; w + 1 < copies; w += 2) {
      t[0] += (double)q[w * plane];
      t[1] += (double)q[(w + 1) * plane];
    }
    if (copies & 1) t[0] += (double)q[(copies - 1) * plane];
    if (!only) pg[c] = first ? t[0] + t[1] : pg[c] + (t[0] + t[1]);
    else if (a.dgamma) store_param(a.dgamma, a.gamma_dt, c, t[0] + t[1]);
  };
#pragma unroll
  for (int k = 0; k < E; k += PER) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      float u = e & 1 ? dg[(k + e) / 2].y : dg[(k + e) / 2].x;
      for (int o = p.seg(); o < 32; o <<= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
      if (!shares_warp(MODE) || ((int)threadIdx.x & 31) < p.L) sh[copy * plane + e * stride + p.lane] = u;
    }
    __syncthreads();
    // neighbouring threads take neighbouring columns
    if constexpr (RAGGED) {
      for (int e = p.mine; e < PER; e += w.rows) add(e, p.lane, column<V, E, true, MODE>(p.L, p.lane, k + e));
    } else {
#pragma unroll
      for (int v = 0; v < PER; v += V)
        for (int j = threadIdx.x; j < V * p.L; j += blockDim.x) add(v + j % V, j / V, (k + v) * p.L + j);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dg[i] = f2(0.0f);
}

// RES: the stored sum has a gradient of its own, read after the row's sum.
// A CTA's share of the rows is fixed, so that the column sums are added in the same order every time. Measured: 32768
// x 8192 bf16 with a residual 322 us (6.7 TB/s), 16384 x 4096 84 (6.4), 100003 x 255 binary32 53 (5.75), 4096 x 16384
// bf16 by clusters of 2 88 (6.1), 4096 x 20480 by clusters of 8 120 (5.6). Bound by memory, in clusters by a step's
// latency, and in short calls by the second kernel (2 to 4 us). Stages of the ring: binary32 2 (3: 100003 x 255 59 us
// instead of 57, 16384 x 2048 68 instead of 66), 16 bits 3 (4 and 5: 1% more).
template <typename T, int MODE, bool RAGGED, bool RES>
__global__ void __launch_bounds__(kBlock, 1) rms_bwd_kernel(RmsGradArgs a) {
  constexpr bool CLUSTER = in_cluster(MODE), GROUP = in_warps(MODE);
  using Mine = Share<MODE>;
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int E = kBwdElems, P = E / 2;
  constexpr int S = rms_bwd_stages<T>(), TN = RES ? 3 : 2;
  __shared__ std::conditional_t<CLUSTER, Meet[kClusterMost], float[2][kBlock / 32]> red;
  extern __shared__ __align__(128) unsigned char dyn[];
  pdl_prologue();
  const Place<MODE> p(a.w.L);
  if (dynamic_smem_bytes() < rms_bwd_smem<T>((int)blockDim.x, p.L, RAGGED, RES)) return;
  float *sh = reinterpret_cast<float *>(dyn + rms_bwd_ring<T>((int)blockDim.x, p.L, RAGGED, RES));
  const int col0 = Mine::first(a.cols);
  double *const parts = a.parts + Mine::unit() * a.w.N + col0;
  ShareWalk<MODE> w = a.w;
  if constexpr (CLUSTER) {
    cut(w, col0, a.cols, RAGGED ? 1 : V);
    red[p.mine].init(p.lane, p.L);
    cluster_sync();
  }
  const int N = (int)w.N;
  const T *src[TN];
  int64_t ld[TN];
  src[0] = static_cast<const T *>(a.h) + col0;
  ld[0] = a.ldh;
  src[1] = static_cast<const T *>(a.dy) + col0;
  ld[1] = a.lddy;
  if constexpr (RES) {
    src[2] = static_cast<const T *>(a.dres) + col0;
    ld[2] = a.lddr;
  }
  const int64_t r0 = (int64_t)Mine::unit() * w.rows;
  int64_t row = r0 + p.mine;
  const int steps = row_count(w.M, r0, w.step), left = row_count(w.M, row, w.step);  // the CTA's, this row's
  RowFeed<T, E, TN, S, RAGGED, MODE> feed(dyn, src, ld, p, w, row);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) feed.issue(p, w, i < left, row + (int64_t)i * w.step);
  // The next row's factor, loaded one row ahead; past its last row a lane stays at that row (at M - 1 if it has none).
  int64_t stat = left > 0 ? row : w.M - 1;
  float next = a.rstd[stat];
  float2 gam[P], dg[P];
  load_pairs<V, E, RAGGED, MODE>(param_from(a.gamma, a.gamma_dt, col0), a.gamma_dt, p, N, 1.0f, gam);
#pragma unroll
  for (int i = 0; i < P; ++i) dg[i] = f2(0.0f);
  const float inv_n = w.inv_n;
  const int warps = GROUP ? p.L / 32 : 1, wl = (int)threadIdx.x & 31, w0 = GROUP ? p.mine * warps : 0;
  char *out = reinterpret_cast<char *>(static_cast<T *>(a.dx) + row * a.lddx + col0);
  bool first = true, lost = false;  // (lost: the others' sums did not come, which the hardware does not let happen)
  int run = 0;
#pragma unroll 1
  for (int it = 0; it < steps; ++it) {
    const bool in = it < left;
    const float rstd = in ? next : 0.0f;
    if (!shares_warp(MODE) && !in) break;  // whole warps without a row: only at the CTA's last step
    feed.wait();
    float2 n[P], d[P];
    feed.read(0, src[0], ld[0], row, p, w, n);
    feed.read(1, src[1], ld[1], row, p, w, d);
    feed.issue(p, w, it + S - 1 < left, row + (int64_t)(S - 1) * w.step);
    if (it + 1 < left) stat += w.step;
    next = a.rstd[stat];
    // Past the row's end n, d and gamma are 0: nothing there enters a sum that is used.
    float2 s[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      n[i] = mul2(n[i], f2(rstd));
      dg[i] = fma2(d[i], n[i], dg[i]);
      d[i] = mul2(gam[i], d[i]);
      s[i & 1] = fma2(d[i], n[i], s[i & 1]);
    }
    s[0] = add2(s[0], s[1]);
    float c = s[0].x + s[0].y;
    c = GROUP ? warp_sum(c) : lanes_sum(c, p.L);
    if constexpr (GROUP) {
      const int par = it & 1;
      if constexpr (CLUSTER) {
        const float nan = __int_as_float(0x7FC00000);
        Meet &meet = red[p.mine];
        meet.put(it, lost ? nan : c, p.lane, p.L);
        if (!lost) lost = !meet.wait(it, p.lane, p.L);
        c = lost ? nan : warp_sum(meet.of[par][wl] + meet.of[par][wl + 32]);
      } else {
        if (wl == 0) red[par][w0 + p.lane / 32] = c;
        group_barrier(p.mine, p.L);
        c = lanes_sum((wl & 15) < warps ? red[par][w0 + (wl & 15)] : 0.0f, 16);
      }
    }
    if (!shares_warp(MODE) || in) {
      c *= inv_n;
      if constexpr (RES) {
        float2 r[P];
        feed.read(2, src[2], ld[2], row, p, w, r);
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = fma2(f2(rstd), fma2(n[i], f2(-c), d[i]), r[i]);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = mul2(f2(rstd), fma2(n[i], f2(-c), d[i]));
      }
      store_pairs<T, E, RAGGED>(reinterpret_cast<T *>(out), d, p, feed, w.NV, N);
    }
    feed.advance(w);
    row += w.step;
    out += a.inc_dx;
    if (++run == kRunRows && it + 1 < steps) {
      rms_flush<V, E, V, RAGGED>(a, parts, w, dg, p, first, sh);
      first = false;
      run = 0;
    }
  }
  // The last run, all elements at once where the ring was: every warp of the
  // CTA is here, also one that left at the last step.
  cp_async_wait<0>();
  __syncthreads();
  rms_flush<V, E, E, RAGGED>(a, parts, w, dg, p, first, reinterpret_cast<float *>(dyn));
  if constexpr (CLUSTER) cluster_sync();  // a CTA ends behind what the others send it
}

// ---- backward: rows too long for registers ---------------------------------------

// c of each row, one CTA per row. (The rows are then read once more: 1024 x 65536 bf16 with a residual 234 us for both
// kernels, 2.3 TB/s of what one pass would move.)
template <typename T, int V>
__global__ void __launch_bounds__(1024) rms_bwd_rows_kernel(RmsGradArgs a, float *cs) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][kMaxWarps];
  pdl_prologue();
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.w.M; row += gridDim.x, par ^= 1) {
    const T *h = static_cast<const T *>(a.h) + row * a.ldh;
    const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
    const float rstd = a.rstd[row];
    float c[1] = {0.0f};
#pragma unroll 2
    for (int64_t cv = threadIdx.x; cv < a.w.NV; cv += blockDim.x) {
      float v[V], d[V], g[V];
      IO::unpack(load_row<T, V>(h + cv * V), v);
      IO::unpack(load_row<T, V>(dy + cv * V), d);
      load_columns<V>(a.gamma, a.gamma_dt, cv * V, 1.0f, g);
#pragma unroll
      for (int e = 0; e < V; ++e) c[0] = fmaf(g[e] * d[e], v[e] * rstd, c[0]);
    }
    cta_sum(c, red[par]);
    if (threadIdx.x == 0) cs[row] = c[0] * a.w.inv_n;
  }
}

// dx and the column sums: a CTA takes blockDim.x vector-columns (blockIdx.x)
// of every gridDim.y-th row.
template <typename T, int V, bool RES>
__global__ void __launch_bounds__(256) rms_bwd_columns_kernel(RmsGradArgs a, const float *cs) {
  using IO = VecIO<T, V>;
  pdl_prologue();
  const int64_t cv = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (cv >= a.w.NV) return;
  const T *h = static_cast<const T *>(a.h) + cv * V;
  const T *dy = static_cast<const T *>(a.dy) + cv * V;
  const T *dr = static_cast<const T *>(a.dres) + (RES ? cv * V : 0);
  T *dx = static_cast<T *>(a.dx) + cv * V;
  float g[V], dg[V];
  load_columns<V>(a.gamma, a.gamma_dt, cv * V, 1.0f, g);
  double sg[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sg[e] = 0.0;
    dg[e] = 0.0f;
  }
  int run = 0;
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < a.w.M; row += gridDim.y) {
    float v[V], d[V], r[V], o[V];
    IO::unpack(load_row<T, V>(h + row * a.ldh), v);
    IO::unpack(load_row<T, V>(dy + row * a.lddy), d);
    if constexpr (RES) IO::unpack(load_row<T, V>(dr + row * a.lddr), r);
    const float rstd = a.rstd[row], c = cs[row];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float n = v[e] * rstd;
      dg[e] = fmaf(d[e], n, dg[e]);
      const float t = fmaf(n, -c, g[e] * d[e]);
      o[e] = RES ? fmaf(rstd, t, r[e]) : rstd * t;
    }
    store_row<T, V>(dx + row * a.lddx, o);
    if (++run == kRunRows) {
      run = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sg[e] += (double)dg[e];
        dg[e] = 0.0f;
      }
    }
  }
  double *pg = a.parts + (int64_t)blockIdx.y * a.w.N + cv * V;
#pragma unroll
  for (int e = 0; e < V; ++e) pg[e] = sg[e] + (double)dg[e];
}

}  // namespace norm
}  // namespace dyt
