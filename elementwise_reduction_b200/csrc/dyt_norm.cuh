// Layer norm forward and backward for sm_100a over the rows of an M x N matrix.
//
//   mean = sum_j x_j / N,  var = sum_j (x_j - mean)^2 / N,  rstd = (var + eps)^-1/2
//   y_j  = gamma_j h_j + beta_j,  h_j = (x_j - mean) rstd
//   dx_j = rstd (g_j - c1 - h_j c2),  g_j = gamma_j dy_j,
//          c1 = sum_j g_j / N,  c2 = sum_j g_j h_j / N
//   dgamma_j = sum_i dy_ij h_ij,  dbeta_j = sum_i dy_ij
//
// Both are bound by memory: a row is read once and kept in registers between
// its sums and its outputs. A row belongs to L lanes: to part of a warp (L a
// power of two up to 32, so that a warp holds 32 / L rows) or to a whole CTA.
// Lane l owns the vectors l, l + L, ... (K of them) of V elements, the same
// columns in every row, so gamma and beta are read once and the column sums of
// the backward stay in registers. V is 16 bytes when every tensor's rows are
// whole aligned vectors, else one element.
#pragma once

#include "dyt_kernels.cuh"

namespace dyt {
namespace norm {

struct NormArgs {
  const void *x;
  int64_t ldx;
  const void *gamma;  // NULL: 1
  const void *beta;   // NULL: 0
  void *y;
  int64_t ldy;
  float *mean;  // NULL: not written
  float *rstd;
  int64_t M;
  int64_t N;
  int NV;  // vectors of a row
  int L;   // lanes of a row (blockDim.x when a CTA has one row)
  int gamma_dt, beta_dt;
  float eps;
};

struct NormGradArgs {
  const void *x;
  int64_t ldx;
  const void *dy;
  int64_t lddy;
  const void *gamma;  // NULL: 1
  const float *mean;
  const float *rstd;
  void *dx;
  int64_t lddx;
  double *parts;  // [CTA][dgamma, dbeta][N] column sums
  int64_t M;
  int64_t N;
  int NV;
  int L;
  int gamma_dt;
};

// Rows a lane adds in binary32 before its column sums move to binary64: the
// run's rounding is at most 128 * 2^-24 of the sum of its terms' magnitudes.
constexpr int kRunRows = 128;
constexpr int kMaxWarps = 32;

// V elements of T at p as stored: one element or 16 bytes.
template <typename T, int V>
__device__ __forceinline__ typename VecIO<T, V>::Raw load_row(const T *p) {
  if constexpr (V == 1) {
    return *p;
  } else {
    return *reinterpret_cast<const uint4 *>(p);
  }
}

// V binary32 values rounded once to T and stored at p.
template <typename T, int V>
__device__ __forceinline__ void store_row(T *p, const float (&f)[V]) {
  using IO = VecIO<T, V>;
  if constexpr (V == 1) {
    IO::store_raw(p, IO::pack(f));
  } else {
    float2 f2[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f2[i] = make_float2(f[2 * i], f[2 * i + 1]);
    IO::store_raw(p, IO::pack2(f2));
  }
}

// gamma or beta at columns c0 .. c0 + V - 1 (a NULL parameter is `none`).
template <int V>
__device__ __forceinline__ void load_columns(const void *p, int dt, int64_t c0, float none, float (&out)[V]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = none;
    return;
  }
  int64_t col[V];
#pragma unroll
  for (int e = 0; e < V; ++e) col[e] = c0 + e;
  load_params<V, void>(p, dt, col, 1.0f, out);
}

// Sums over the lanes of a row. Part of a warp: a butterfly, every lane gets
// the same bits. A CTA: the warps' sums meet in shared memory (`red`, a buffer
// that the call before the last one may still be read from), one barrier.
template <bool CTA, int C>
__device__ __forceinline__ void row_sum(float (&v)[C], int L, float *red) {
  if constexpr (!CTA) {
    for (int o = L >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] += __shfl_xor_sync(0xFFFFFFFFu, v[c], o);
    }
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] += __shfl_xor_sync(0xFFFFFFFFu, v[c], o);
    }
    if (lane == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) red[c * kMaxWarps + warp] = v[c];
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = lane < warps ? red[c * kMaxWarps + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] += __shfl_xor_sync(0xFFFFFFFFu, v[c], o);
    }
  }
}

// ---- forward: a row in registers ---------------------------------------------

template <typename T, int V, int K, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : 256) norm_fwd_kernel(NormArgs a) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][kMaxWarps];
  pdl_prologue();
  const int L = CTA ? (int)blockDim.x : a.L;
  const int lane = CTA ? (int)threadIdx.x : (int)threadIdx.x & (L - 1);
  const int rows = CTA ? 1 : (int)blockDim.x / L;
  const int mine = CTA ? 0 : (int)threadIdx.x / L;
  const T *x = static_cast<const T *>(a.x);
  T *y = static_cast<T *>(a.y);
  float gam[K][V], bet[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int cv = lane + k * L;
    if (cv < a.NV) {
      load_columns<V>(a.gamma, a.gamma_dt, (int64_t)cv * V, 1.0f, gam[k]);
      load_columns<V>(a.beta, a.beta_dt, (int64_t)cv * V, 0.0f, bet[k]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) gam[k][e] = bet[k][e] = 0.0f;
    }
  }
  const float inv_n = 1.0f / (float)a.N;
  const int64_t step = (int64_t)gridDim.x * rows;
  typename IO::Raw next[K];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int cv = lane + k * L;
      next[k] = row < a.M && cv < a.NV ? load_row<T, V>(x + row * a.ldx + (int64_t)cv * V) : typename IO::Raw{};
    }
  };
  int64_t r0 = (int64_t)blockIdx.x * rows;  // every thread of a CTA makes the same steps
  fetch(r0 + mine);
  for (; r0 < a.M; r0 += step) {
    const int64_t row = r0 + mine;
    float v[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) IO::unpack(next[k], v[k]);
    fetch(row + step);
    float s[1] = {0.0f};  // the vectors past a row's end are zero
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] += v[k][e];
    row_sum<CTA, 1>(s, L, red[0]);
    const float mean = s[0] / (float)a.N;  // exact for a constant row
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = lane + k * L < a.NV;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[k][e] = in ? v[k][e] - mean : 0.0f;
        q[0] = fmaf(v[k][e], v[k][e], q[0]);
      }
    }
    row_sum<CTA, 1>(q, L, red[1]);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv_n, a.eps));
    if (row < a.M) {
      if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int cv = lane + k * L;
        if (cv < a.NV) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = fmaf(v[k][e] * rstd, gam[k][e], bet[k][e]);
          store_row<T, V>(y + row * a.ldy + (int64_t)cv * V, o);
        }
      }
    }
  }
}

// ---- forward: rows too long for registers --------------------------------------

// One CTA reads each row three times (the second and third time mostly from
// L2): its sum, its centred squares, its outputs.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(NormArgs a) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][kMaxWarps];
  pdl_prologue();
  const float inv_n = 1.0f / (float)a.N;
  const int B = blockDim.x;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    T *y = static_cast<T *>(a.y) + row * a.ldy;
    float s[1] = {0.0f};
#pragma unroll 4
    for (int64_t cv = threadIdx.x; cv < a.NV; cv += B) {
      float v[V];
      IO::unpack(load_row<T, V>(x + cv * V), v);
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] += v[e];
    }
    row_sum<true, 1>(s, B, red[0]);
    const float mean = s[0] / (float)a.N;  // exact for a constant row
    float q[1] = {0.0f};
#pragma unroll 4
    for (int64_t cv = threadIdx.x; cv < a.NV; cv += B) {
      float v[V];
      IO::unpack(load_row<T, V>(x + cv * V), v);
#pragma unroll
      for (int e = 0; e < V; ++e) q[0] = fmaf(v[e] - mean, v[e] - mean, q[0]);
    }
    row_sum<true, 1>(q, B, red[1]);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv_n, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t cv = threadIdx.x; cv < a.NV; cv += B) {
      float v[V], g[V], b[V];
      IO::unpack(load_row<T, V>(x + cv * V), v);
      load_columns<V>(a.gamma, a.gamma_dt, cv * V, 1.0f, g);
      load_columns<V>(a.beta, a.beta_dt, cv * V, 0.0f, b);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = fmaf((v[e] - mean) * rstd, g[e], b[e]);
      store_row<T, V>(y + cv * V, v);
    }
  }
}

// ---- backward: a row in registers ------------------------------------------------

// A lane's column sums of one run of rows, moved to the CTA's partial sums in
// binary64 (added to them after the first run). Rows side by side in a warp
// are added by a butterfly over the lanes that own the same columns, the warps
// in order.
template <int V, int K, bool CTA>
__device__ __forceinline__ void flush_columns(const NormGradArgs &a, float (&dg)[K][V], float (&db)[K][V], int lane,
                                              int L, bool first, float *sh) {
  double *pg = a.parts + (int64_t)blockIdx.x * 2 * a.N, *pb = pg + a.N;
  if constexpr (CTA) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int cv = lane + k * L;
      if (cv < a.NV) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int64_t c = (int64_t)cv * V + e;
          pg[c] = first ? (double)dg[k][e] : pg[c] + (double)dg[k][e];
          pb[c] = first ? (double)db[k][e] : pb[c] + (double)db[k][e];
        }
      }
    }
  } else {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int width = L * K * V;  // columns, padded
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = dg[k][e], w = db[k][e];
        for (int o = L; o < 32; o <<= 1) {
          u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
          w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
        }
        if ((threadIdx.x & 31) < L) {
          const int c = (lane + k * L) * V + e;
          sh[(warp * 2) * width + c] = u;
          sh[(warp * 2 + 1) * width + c] = w;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += blockDim.x) {
      const int which = i >= width, c = i - which * width;
      if (c < a.N) {
        double t = 0.0;
        for (int w = 0; w < warps; ++w) t += (double)sh[(w * 2 + which) * width + c];
        double *p = which ? pb : pg;
        p[c] = first ? t : p[c] + t;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) dg[k][e] = db[k][e] = 0.0f;
}

template <typename T, int V, int K, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : 256) norm_bwd_kernel(NormGradArgs a) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][2 * kMaxWarps];
  extern __shared__ float sh[];  // rows side by side: [warp][dgamma, dbeta][L K V]
  pdl_prologue();
  const int L = CTA ? (int)blockDim.x : a.L;
  const int lane = CTA ? (int)threadIdx.x : (int)threadIdx.x & (L - 1);
  const int rows = CTA ? 1 : (int)blockDim.x / L;
  const int mine = CTA ? 0 : (int)threadIdx.x / L;
  const T *x = static_cast<const T *>(a.x);
  const T *dy = static_cast<const T *>(a.dy);
  T *dx = static_cast<T *>(a.dx);
  float gam[K][V], dg[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int cv = lane + k * L;
#pragma unroll
    for (int e = 0; e < V; ++e) gam[k][e] = dg[k][e] = db[k][e] = 0.0f;
    if (cv < a.NV) load_columns<V>(a.gamma, a.gamma_dt, (int64_t)cv * V, 1.0f, gam[k]);
  }
  const float inv_n = 1.0f / (float)a.N;
  const int64_t step = (int64_t)gridDim.x * rows;
  typename IO::Raw nx[K], nd[K];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int64_t row) {
    const bool in = row < a.M;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int cv = lane + k * L;
      nx[k] = in && cv < a.NV ? load_row<T, V>(x + row * a.ldx + (int64_t)cv * V) : typename IO::Raw{};
      nd[k] = in && cv < a.NV ? load_row<T, V>(dy + row * a.lddy + (int64_t)cv * V) : typename IO::Raw{};
    }
    nmean = in ? a.mean[row] : 0.0f;
    nrstd = in ? a.rstd[row] : 0.0f;
  };
  int64_t r0 = (int64_t)blockIdx.x * rows;
  fetch(r0 + mine);
  bool first = true;
  int run = 0, par = 0;
  for (; r0 < a.M; r0 += step) {
    const int64_t row = r0 + mine;
    float h[K][V], d[K][V];
    const float mean = nmean, rstd = nrstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      IO::unpack(nx[k], h[k]);
      IO::unpack(nd[k], d[k]);
    }
    fetch(row + step);
    float c[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = row < a.M && lane + k * L < a.NV;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        h[k][e] = in ? (h[k][e] - mean) * rstd : 0.0f;
        dg[k][e] = fmaf(d[k][e], h[k][e], dg[k][e]);
        db[k][e] += d[k][e];
        const float g = gam[k][e] * d[k][e];
        c[0] += g;
        c[1] = fmaf(g, h[k][e], c[1]);
        d[k][e] = g;
      }
    }
    row_sum<CTA, 2>(c, L, red[par]);
    par ^= 1;
    const float c1 = c[0] * inv_n, c2 = c[1] * inv_n;
    if (row < a.M) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int cv = lane + k * L;
        if (cv < a.NV) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = rstd * (d[k][e] - fmaf(h[k][e], c2, c1));
          store_row<T, V>(dx + row * a.lddx + (int64_t)cv * V, o);
        }
      }
    }
    if (++run == kRunRows) {
      flush_columns<V, K, CTA>(a, dg, db, lane, L, first, sh);
      first = false;
      run = 0;
    }
  }
  if (run > 0 || first) flush_columns<V, K, CTA>(a, dg, db, lane, L, first, sh);
}

// ---- backward: rows too long for registers ------------------------------------------

// c1 and c2 of each row, one CTA per row.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_bwd_rows_kernel(NormGradArgs a, float2 *c12) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][2 * kMaxWarps];
  pdl_prologue();
  const float inv_n = 1.0f / (float)a.N;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, par ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int64_t cv = threadIdx.x; cv < a.NV; cv += blockDim.x) {
      float v[V], d[V], g[V];
      IO::unpack(load_row<T, V>(x + cv * V), v);
      IO::unpack(load_row<T, V>(dy + cv * V), d);
      load_columns<V>(a.gamma, a.gamma_dt, cv * V, 1.0f, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float gd = g[e] * d[e];
        c[0] += gd;
        c[1] = fmaf(gd, (v[e] - mean) * rstd, c[1]);
      }
    }
    row_sum<true, 2>(c, (int)blockDim.x, red[par]);
    if (threadIdx.x == 0) c12[row] = make_float2(c[0] * inv_n, c[1] * inv_n);
  }
}

// dx and the column sums: a CTA takes blockDim.x vector-columns (blockIdx.x)
// of every gridDim.y-th row.
template <typename T, int V>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(NormGradArgs a, const float2 *__restrict__ c12) {
  using IO = VecIO<T, V>;
  pdl_prologue();
  const int64_t cv = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (cv >= a.NV) return;
  const T *x = static_cast<const T *>(a.x) + cv * V;
  const T *dy = static_cast<const T *>(a.dy) + cv * V;
  T *dx = static_cast<T *>(a.dx) + cv * V;
  float g[V];
  load_columns<V>(a.gamma, a.gamma_dt, cv * V, 1.0f, g);
  double sg[V], sb[V];
  float dg[V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sg[e] = sb[e] = 0.0;
    dg[e] = db[e] = 0.0f;
  }
  int run = 0;
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
    float v[V], d[V], o[V];
    IO::unpack(load_row<T, V>(x + row * a.ldx), v);
    IO::unpack(load_row<T, V>(dy + row * a.lddy), d);
    const float mean = a.mean[row], rstd = a.rstd[row];
    const float2 c = c12[row];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float h = (v[e] - mean) * rstd;
      dg[e] = fmaf(d[e], h, dg[e]);
      db[e] += d[e];
      o[e] = rstd * (g[e] * d[e] - fmaf(h, c.y, c.x));
    }
    store_row<T, V>(dx + row * a.lddx, o);
    if (++run == kRunRows) {
      run = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sg[e] += (double)dg[e];
        sb[e] += (double)db[e];
        dg[e] = db[e] = 0.0f;
      }
    }
  }
  double *pg = a.parts + (int64_t)blockIdx.y * 2 * a.N + cv * V, *pb = pg + a.N;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    pg[e] = sg[e] + (double)dg[e];
    pb[e] = sb[e] + (double)db[e];
  }
}

// ---- backward: the parameters' gradients ---------------------------------------------

constexpr int kSumCols = 32, kSumLanes = 8;

// The CTAs' column sums added in binary64 in a fixed order (lane l takes
// partials l, l + 8, ...; the lanes are added in order) and rounded once.
// blockIdx.y: 0 = dgamma, 1 = dbeta.
__global__ void __launch_bounds__(kSumCols *kSumLanes)
    norm_finalize_kernel(const double *__restrict__ parts, int nparts, int64_t N, void *dgamma, int gamma_dt,
                         void *dbeta, int beta_dt) {
  __shared__ double sh[kSumLanes][kSumCols];
  pdl_prologue();
  const int c = threadIdx.x & (kSumCols - 1), lane = threadIdx.x / kSumCols;
  const int64_t col = (int64_t)blockIdx.x * kSumCols + c;
  void *out = blockIdx.y ? dbeta : dgamma;
  if (out == nullptr) return;
  double t = 0.0;
  if (col < N) {
    const double *p = parts + blockIdx.y * N + col;
#pragma unroll 4
    for (int i = lane; i < nparts; i += kSumLanes) t += p[(int64_t)i * 2 * N];
  }
  sh[lane][c] = t;
  __syncthreads();
  if (lane == 0 && col < N) {
    double s = 0.0;
#pragma unroll
    for (int l = 0; l < kSumLanes; ++l) s += sh[l][c];
    store_param(out, blockIdx.y ? beta_dt : gamma_dt, col, s);
  }
}

}  // namespace norm
}  // namespace dyt
