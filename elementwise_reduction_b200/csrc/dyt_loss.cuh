// The clipped policy loss with a KL term, forward and backward, for sm_100a,
// from the logits of M rows (tokens) over a vocabulary of N.
//
//   m = max_j z_j,  s = log sum_j exp((z_j - m) / T),  lp = (z_t - m) / T - s
//   r = exp(lp - old),  c = clip(r, 1 - lo, 1 + hi),  q = ref - lp
//   loss = sum_i w_i (-min(r A, c A) + kl (exp(q) - q - 1))
//   coef = w (-(r A where r A <= c A, else 0) + kl (1 - exp(q)))   (d loss / d lp)
//   dz_j = (grad coef / T) ([j = t] - exp((z_j - m) / T - s))
//
// Both passes are bound by reading (and writing) the logits once. The forward
// keeps a running maximum and sum per thread; rows are split over several CTAs
// when there are few of them, and the second kernel joins the parts, does the
// rows' scalar arithmetic in binary64 and adds the loss in a fixed order. Rows
// of weight 0 are not read.
//
// Exponentials are 2^((z - m) C) with C = log2(e) / T in binary32: the maximum is
// taken out before anything is rounded to its size, and its own term is exactly 1.
#pragma once

#include <cooperative_groups.h>

#include "dyt_kernels.cuh"

namespace dyt {
namespace loss {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr double kLn2 = 0.693147180559945309417232121458;
constexpr double kLog2eD = 1.44269504088896340735992468100;

struct LossArgs {
  const void *z;
  int64_t ld;
  const void *tokens;  // int64 or int32 (wide_tokens)
  const float *old_logp;
  const float *ref_logp;   // NULL: no KL term
  const float *advantage;
  const float *weight;     // NULL: 1 / M
  float *loss;             // [1]
  float *logp;             // [M]
  float2 *stats;           // [M] (m, s)
  float *coef;             // [M]
  float2 *parts;           // [M][S] (maximum, sum of 2^((z - maximum) C)) of each part of a row
  int64_t M;
  int64_t N;
  int S;                   // parts of a row
  int wide_tokens;
  float C;                 // log2(e) / T
  double inv_t;
  double lo, hi;           // 1 - clip_low, 1 + clip_high
  double kl;
};

struct LossGradArgs {
  const void *z;
  int64_t ld;
  const void *tokens;
  const float2 *stats;
  const float *coef;
  const float *grad;  // NULL: 1
  void *dz;
  int64_t lddz;
  int64_t M;
  int64_t N;
  int S;
  int wide_tokens;
  float C;
  double inv_t;
};

__device__ __forceinline__ int64_t token_at(const void *p, int wide, int64_t row) {
  return wide ? static_cast<const int64_t *>(p)[row] : (int64_t) static_cast<const int32_t *>(p)[row];
}

// ---- running maximum and sum -----------------------------------------------------

struct Run {
  float m = kNegInf;  // largest logit so far
  float s = 0.0f;     // sum of 2^((z - m) C)
};

__device__ __forceinline__ Run join(const Run &a, const Run &b, float C) {
  Run r;
  r.m = fmaxf(a.m, b.m);
  // Equal maxima keep their sum as it is (infinities included).
  r.s = (a.m == r.m ? a.s : a.s * ex2_approx((a.m - r.m) * C)) + (b.m == r.m ? b.s : b.s * ex2_approx((b.m - r.m) * C));
  return r;
}

// 2 n values more. NaN passes over the maximum and reaches the sum.
template <int n>
__device__ __forceinline__ void add_pairs(Run &r, const float2 (&v)[n], float C) {
  float2 t = v[0];
#pragma unroll
  for (int i = 1; i < n; ++i) t = make_float2(fmaxf(t.x, v[i].x), fmaxf(t.y, v[i].y));
  const float top = fmaxf(t.x, t.y);
  if (top > r.m) {
    r.s *= ex2_approx((r.m - top) * C);  // 0 for the first values: 2^-inf
    r.m = top;
  }
  const float m = r.m == kNegInf ? 0.0f : r.m;  // only -inf so far: every term is 2^-inf
  float2 s[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float2 e = mul2(add2(v[i], f2(-m)), f2(C));
    s[i & 1] = add2(s[i & 1], make_float2(ex2_approx(e.x), ex2_approx(e.y)));
  }
  s[0] = add2(s[0], s[1]);
  r.s += s[0].x + s[0].y;
}

__device__ __forceinline__ void add_one(Run &r, float v, float C) {
  const float2 p[1] = {make_float2(v, kNegInf)};
  add_pairs(r, p, C);
}

template <typename T>
__device__ __forceinline__ int head_elems(const T *p, int64_t N) {
  const int h = (int)((16u - (uint32_t)((uintptr_t)p & 15u)) & 15u) / (int)sizeof(T);
  return h < N ? h : (int)N;
}

// One part of one row per G threads (a warp, or the CTA): the row's whole
// 16-byte vectors are cut into S parts, its first and last elements off those
// vectors go with the first and the last part.
template <typename T, bool CTA>
__global__ void __launch_bounds__(256) loss_rows_kernel(LossArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int U = 4;
  using IO = VecIO<T, V>;
  __shared__ Run sh[8];
  pdl_prologue();
  const int G = CTA ? (int)blockDim.x : 32;
  const int t = CTA ? (int)threadIdx.x : (int)threadIdx.x & 31;
  const int64_t items = a.M * a.S;
  const int64_t step = CTA ? gridDim.x : (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t item = CTA ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  for (; item < items; item += step) {
    const int64_t row = a.S == 1 ? item : item / a.S;
    const int part = (int)(item - row * a.S);
    if (a.weight && a.weight[row] == 0.0f) continue;
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    const int head = head_elems(z, a.N);
    const int64_t nb = (a.N - head) / V;
    const int tail = (int)(a.N - head - nb * V);
    const int64_t b0 = nb * part / a.S, b1 = nb * (part + 1) / a.S;
    Run r;
    if (part == 0 && t < head) add_one(r, to_f32<T>(z[t]), a.C);
    if (part == a.S - 1 && t < tail) add_one(r, to_f32<T>(z[a.N - tail + t]), a.C);
    const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);
    int64_t i = b0 + t;
    for (; i + (U - 1) * G < b1; i += U * G) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = __ldcs(zv + i + u * G);
      float2 v[U * V / 2];
#pragma unroll
      for (int u = 0; u < U; ++u) IO::unpack2(raw[u], *reinterpret_cast<float2(*)[V / 2]>(v + u * V / 2));
      add_pairs(r, v, a.C);
    }
    for (; i < b1; i += G) {
      float2 v[V / 2];
      IO::unpack2(__ldcs(zv + i), v);
      add_pairs(r, v, a.C);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Run other;
      other.m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o);
      other.s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
      // the lower lane's part first, on both sides: the same bits
      r = (threadIdx.x & o) ? join(other, r, a.C) : join(r, other, a.C);
    }
    if constexpr (CTA) {
      if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = r;
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int w = 1; w < G / 32; ++w) r = join(r, sh[w], a.C);
      }
      __syncthreads();
    }
    if (t == 0) a.parts[item] = make_float2(r.m, r.s);
  }
}

// What row i adds to the loss; writes its outputs.
template <typename T>
__device__ __forceinline__ double finish_row(const LossArgs &a, int64_t row, const Run &r, double w) {
  const T *z = static_cast<const T *>(a.z) + row * a.ld;
  const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
  // a token outside the vocabulary has no probability: NaN, here and in the loss
  const double hit = tok >= 0 && tok < a.N ? (double)to_f32<T>(z[tok]) : (double)__int_as_float(0x7FC00000);
  const double s = log((double)r.s);
  const double lp = (hit - (double)r.m) * a.inv_t - s;
  const double A = (double)a.advantage[row];
  const double ratio = exp(lp - (double)a.old_logp[row]);
  const double ra = ratio * A, ca = fmin(fmax(ratio, a.lo), a.hi) * A;
  const bool held = ra > ca;  // the clipped side is the smaller one: no gradient
  double each = held ? -ca : -ra, d = held ? 0.0 : -ra;
  if (a.ref_logp && a.kl != 0.0) {
    const double q = (double)a.ref_logp[row] - lp, em = expm1(q);
    each += a.kl * (em - q);
    d -= a.kl * em;
  }
  a.logp[row] = (float)lp;
  a.stats[row] = make_float2(r.m, (float)s);
  a.coef[row] = (float)(w * d);
  return w * each;
}

// Joins the rows' parts, finishes the rows and adds the loss: one cluster, a
// thread per row (S = 1) or a warp per row, each CTA's sum added in order.
template <typename T>
__global__ void __launch_bounds__(512) loss_finish_kernel(LossArgs a) {
  namespace cg = cooperative_groups;
  __shared__ double sh[16];
  __shared__ double total;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)gridDim.x, tid = threadIdx.x;
  double sum = 0.0;
  const int64_t per = (a.S == 1 ? blockDim.x : blockDim.x / 32);  // rows of a CTA step
  for (int64_t row = (int64_t)blockIdx.x * per + (a.S == 1 ? tid : tid >> 5); row < a.M; row += per * ctas) {
    const double w = a.weight ? (double)a.weight[row] : 1.0 / (double)a.M;
    Run r;
    if (w != 0.0) {
      if (a.S == 1) {
        const float2 p = a.parts[row];
        r.m = p.x;
        r.s = p.y;
      } else {
        for (int i = tid & 31; i < a.S; i += 32) {
          const float2 p = a.parts[row * a.S + i];
          Run o;
          o.m = p.x;
          o.s = p.y;
          r = join(r, o, a.C);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          Run other;
          other.m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o);
          other.s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
          r = (tid & o) ? join(other, r, a.C) : join(r, other, a.C);
        }
      }
    }
    if (a.S == 1 || (tid & 31) == 0) {
      if (w != 0.0) {
        sum += finish_row<T>(a, row, r, w);
      } else {
        a.logp[row] = 0.0f;
        a.stats[row] = make_float2(0.0f, 0.0f);
        a.coef[row] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((tid & 31) == 0) sh[tid >> 5] = sum;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += sh[w];
    total = s;
  }
  cluster.sync();
  if (blockIdx.x == 0 && tid == 0) {
    double s = 0.0;
    for (int c = 0; c < ctas; ++c) s += *cluster.map_shared_rank(&total, c);
    *a.loss = (float)s;
  }
  cluster.sync();  // every CTA's shared memory stays until it has been read
}

// ---- backward -------------------------------------------------------------------------

// 16 bytes at p, d bytes past a 16-byte boundary (whole elements), from the
// two aligned vectors that hold them.
__device__ __forceinline__ uint4 cut16(const uint4 &lo, const uint4 &hi, uint32_t d) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (d & 8u) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (d & 4u) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t b = (d & 3u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], b), __funnelshift_r(w[1], w[2], b), __funnelshift_r(w[2], w[3], b),
                    __funnelshift_r(w[3], w[4], b));
}

// G threads (a warp, or the CTA) per part of a row. The vectors are those of
// the output row; SHIFT: the input row lies at another offset past a 16-byte
// boundary, and each of its vectors is cut out of two aligned ones inside the
// row. The elements before and after those vectors are taken one by one.
template <typename T, bool CTA, bool SHIFT>
__global__ void __launch_bounds__(256) loss_grad_kernel(LossGradArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int U = SHIFT ? 2 : 4;
  using IO = VecIO<T, V>;
  pdl_prologue();
  const int G = CTA ? (int)blockDim.x : 32;
  const int t = CTA ? (int)threadIdx.x : (int)threadIdx.x & 31;
  const int64_t items = a.M * a.S;
  const int64_t step = CTA ? gridDim.x : (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t item = CTA ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const double gt = (a.grad ? (double)*a.grad : 1.0) * a.inv_t;
  for (; item < items; item += step) {
    const int64_t row = a.S == 1 ? item : item / a.S;
    const int part = (int)(item - row * a.S);
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    T *dz = static_cast<T *>(a.dz) + row * a.lddz;
    const float A = (float)(gt * (double)a.coef[row]);
    // whole output vectors [head, head + nb V): with SHIFT, those whose two
    // input vectors lie inside the row
    int64_t head = head_elems(dz, a.N);
    int d = 0;
    int64_t nb = (a.N - head) / V;
    if constexpr (SHIFT) {
      d = (int)(((uintptr_t)(z + head) & 15u) / sizeof(T));
      if (d > 0) {
        if (head < d) head += V;
        nb = (a.N - head + d - V) / V;
        if (a.N - head + d < V || head > a.N) nb = 0;
      }
      if (nb == 0) head = 0;
    }
    const int64_t rest = a.N - head - nb * V;  // elements after the vectors
    const int64_t b0 = nb * part / a.S, b1 = nb * (part + 1) / a.S;
    uint4 *out = reinterpret_cast<uint4 *>(dz + head);
    if (A == 0.0f) {  // no weight, or the clipped side: no gradient whatever the logits are
      if (part == 0)
        for (int64_t j = t; j < head; j += G) dz[j] = from_f32<T>(0.0f);
      if (part == a.S - 1)
        for (int64_t j = t; j < rest; j += G) dz[a.N - rest + j] = from_f32<T>(0.0f);
      for (int64_t i = b0 + t; i < b1; i += G) __stcs(out + i, make_uint4(0u, 0u, 0u, 0u));
      continue;
    }
    const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
    const float2 st = a.stats[row];
    // p = 2^(z C - K), K = m C + s log2(e); K's rounding, |k - K| <= 2^-24 |K|,
    // goes into the factor as 1 + (k - K) ln 2 (its square is below 2^-34 for |K| < 100)
    const double K = (double)st.x * (double)a.C + (double)st.y * kLog2eD;
    const float k = (float)K;
    const float B = -A * fmaf((float)((double)k - K), (float)kLn2, 1.0f);
    auto one = [&](int64_t j) {
      const float p = ex2_approx(fmaf(to_f32<T>(z[j]), a.C, -k));
      dz[j] = from_f32<T>(j == tok ? fmaf(B, p, A) : B * p);
    };
    if (part == 0)
      for (int64_t j = t; j < head; j += G) one(j);
    if (part == a.S - 1)
      for (int64_t j = t; j < rest; j += G) one(a.N - rest + j);
    const uint4 *in = reinterpret_cast<const uint4 *>(z + (head - d));
    auto vec = [&](int64_t i, const uint4 &raw) {
      float v[V];
      IO::unpack(raw, v);
      const int64_t j0 = head + i * V;
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = B * ex2_approx(fmaf(v[e], a.C, -k));
      if (tok >= j0 && tok < j0 + V) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += j0 + e == tok ? A : 0.0f;
      }
      float2 f[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) f[e] = make_float2(v[2 * e], v[2 * e + 1]);
      __stcs(out + i, IO::pack2(f));
    };
    int64_t i = b0 + t;
    for (; i + (U - 1) * G < b1; i += U * G) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = __ldcs(in + i + u * G);
        if constexpr (SHIFT) {
          if (d > 0) raw[u] = cut16(raw[u], in[i + u * G + 1], (uint32_t)d * sizeof(T));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) vec(i + u * G, raw[u]);
    }
    for (; i < b1; i += G) {
      uint4 raw = in[i];
      if constexpr (SHIFT) {
        if (d > 0) raw = cut16(raw, in[i + 1], (uint32_t)d * sizeof(T));
      }
      vec(i, raw);
    }
  }
}

}  // namespace loss
}  // namespace dyt
