// The clipped policy loss with a KL term, forward and backward, for sm_100a,
// from the logits of M rows (tokens) over a vocabulary of N.
//
//   m = max_j z_j,  s = log sum_j exp((z_j - m) / T),  lp = (z_t - m) / T - s
//   r = exp(lp - old),  c = clip(r, 1 - lo, 1 + hi),  q = ref - lp
//   loss = sum_i w_i (-min(r A, c A) + kl (exp(q) - q - 1))
//   coef = w (-(r A where r A <= c A, else 0) + kl (1 - exp(q)))   (d loss / d lp)
//   dz_j = (grad coef / T) ([j = t] - exp((z_j - m) / T - s))
//
// Both passes are bound by reading (and writing) the logits once. In the
// forward a warp takes one row, or one of S parts of it, at a time, keeps a
// running maximum and sum per lane, and reads ahead into its next item, so that
// the memory never waits for the end of a row. The second kernel joins the
// parts, does the rows' scalar arithmetic in binary64 and adds the loss in a
// fixed order. Rows of weight 0 are not read.
//
// Exponentials are 2^((z - m) C) with C = log2(e) / T in binary32: the maximum is
// taken out before anything is rounded to its size, and its own term is exactly 1.
#pragma once

#include "dyt_async.cuh"

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
  double *sums;            // [CTA of the second kernel] what its rows add to the loss
  unsigned *done;          // how many of those CTAs have finished
  int64_t M;
  int64_t N;
  int S;                   // parts of a row
  int part_vecs;           // 16-byte vectors of each, the last one's may be fewer
  int aligned;             // every row is whole aligned 16-byte vectors
  int64_t row_step;        // a warp's next item lies part_step parts and row_step rows further on
  int part_step;
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

// The largest of three (one instruction on sm_100); a NaN passes over.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2 n values more. NaN passes over the maximum and reaches the sum.
template <int n>
__device__ __forceinline__ void add_pairs(Run &r, const float2 (&v)[n], float C) {
  float t[2] = {fmaxf(v[0].x, v[0].y), kNegInf};
#pragma unroll
  for (int i = 1; i < n; ++i) t[i & 1] = max3(t[i & 1], v[i].x, v[i].y);
  const float top = fmaxf(t[0], t[1]);
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

template <typename T>
__device__ __forceinline__ int head_elems(const T *p, int64_t N) {
  const int h = (int)((16u - (uint32_t)((uintptr_t)p & 15u)) & 15u) / (int)sizeof(T);
  return h < N ? h : (int)N;
}

constexpr int kRowsBlock = 256;        // threads of a CTA of the forward, at most
constexpr int kBatch = 8, kStages = 3;  // a lane's 16-byte vectors in a batch, and batches in its ring
constexpr int kQueue = 4;               // items that a warp has begun to read, at most kStages

__host__ __device__ constexpr size_t rows_smem(int block) { return (size_t)block * kBatch * kStages * 16; }

// The items (row, part) a warp reads, all rows' first parts before their second
// ones: item, item + warps, ... without those of weight 0. Weights are looked
// up 32 items at a time, one per lane.
struct Items {
  int64_t row;
  int part;
  uint32_t mask;  // which of the items looked up count, from the current one on
  int left;       // how many of them there are

  __device__ __forceinline__ bool any(const LossArgs &a) const { return part < a.S; }
  __device__ __forceinline__ void load(const LossArgs &a) {
    const int k = threadIdx.x & 31;
    const int64_t r = row + k * a.row_step, over = r / a.M;
    const int64_t p = part + (int64_t)k * a.part_step + over;
    mask = __ballot_sync(0xFFFFFFFFu, p < a.S && (a.weight == nullptr || a.weight[r - over * a.M] != 0.0f));
    left = 32;
  }
  __device__ __forceinline__ void step(const LossArgs &a) {
    row += a.row_step;
    part += a.part_step;
    if (row >= a.M) {
      row -= a.M;
      ++part;
    }
    mask >>= 1;
    if (--left == 0 && any(a)) load(a);
  }
  // To the first item that counts, from the current one on; false: there is none.
  __device__ __forceinline__ bool find(const LossArgs &a) {
    while (any(a) && !(mask & 1u)) step(a);
    return any(a);
  }
};

struct Item {
  int64_t row;
  int part;
  int nv;  // whole 16-byte vectors of the part
};

// A warp's items, one after the other: the row's whole 16-byte vectors are cut
// into S parts, the elements before and after them go with the first and the
// last part. Every lane keeps kStages batches of vectors in a ring of its own
// (asynchronous copies), also across items.
template <typename T>
__global__ void __launch_bounds__(kRowsBlock, 2) loss_rows_kernel(LossArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int P = V / 2;
  using IO = VecIO<T, V>;
  __shared__ Item queue[kRowsBlock / 32][kQueue];
  extern __shared__ __align__(16) unsigned char dyn[];
  pdl_prologue();
  if (dynamic_smem_bytes() < rows_smem((int)blockDim.x)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0u;
  uint4 *ring = reinterpret_cast<uint4 *>(dyn) + warp * (kStages * kBatch * 32) + lane;
  Items it;
  {
    const int64_t first = (int64_t)blockIdx.x * ((int)blockDim.x >> 5) + warp;
    it.part = (int)(first / a.M);
    it.row = first - it.part * a.M;
    it.load(a);
  }
  const uint4 *src = nullptr;  // this lane's next vector of the item being read
  int ahead = 0;               // vectors of it not yet asked for
  int put = 0, wr = 0;         // items begun, the ring's first slot to fill
  bool reading = false;
  auto issue = [&]() {
    if (!reading && it.find(a)) {
      const T *z = static_cast<const T *>(a.z) + it.row * a.ld;
      const int head = a.aligned ? 0 : head_elems(z, a.N);
      const int nb = (int)((a.N - head) / V);
      // cut at whole batches, so that only a row's last one is not full
      const int b0 = min(it.part * a.part_vecs, nb), b1 = it.part == a.S - 1 ? nb : min(b0 + a.part_vecs, nb);
      src = reinterpret_cast<const uint4 *>(z + head) + b0 + lane;
      ahead = b1 - b0;
      if (lane == 0) queue[warp][put % kQueue] = Item{it.row, it.part, ahead};
      __syncwarp();
      ++put;
      reading = true;
      it.step(a);
    }
    if (reading) {
      uint4 *slot = ring + wr;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u * 32 + lane < ahead) cp_async16(slot + u * 32, src + u * 32);
      src += kBatch * 32;
      ahead -= kBatch * 32;
      reading = ahead > 0;
    }
    cp_async_commit();
    wr = wr == (kStages - 1) * kBatch * 32 ? 0 : wr + kBatch * 32;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();
  int rd = 0;
  const float C = a.C;
  for (int got = 0; got < put; ++got) {
    const Item item = queue[warp][got % kQueue];
    // The elements off the vectors: used only after those, so that nothing waits for them.
    float first = kNegInf, last = kNegInf;
    if (!a.aligned) {
      const T *z = static_cast<const T *>(a.z) + item.row * a.ld;
      const int head = head_elems(z, a.N), tail = (int)((a.N - head) % V);
      if (item.part == 0 && lane < head) first = to_f32<T>(z[lane]);
      if (item.part == a.S - 1 && lane < tail) last = to_f32<T>(z[a.N - tail + lane]);
    }
    Run r;
    int n = item.nv;
    do {
      cp_async_wait<kStages - 2>();
      uint4 raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) raw[u] = ring[rd + u * 32];
      rd = rd == (kStages - 1) * kBatch * 32 ? 0 : rd + kBatch * 32;
      issue();
      if (n >= kBatch * 32) {
        float2 v[kBatch * P];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) IO::unpack2(raw[u], *reinterpret_cast<float2(*)[P]>(v + u * P));
        add_pairs(r, v, C);
      } else {
        float2 v[kBatch * P];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          IO::unpack2(raw[u], *reinterpret_cast<float2(*)[P]>(v + u * P));
          if (u * 32 + lane >= n)
#pragma unroll
            for (int i = 0; i < P; ++i) v[u * P + i] = f2(kNegInf);
        }
        add_pairs(r, v, C);
      }
      n -= kBatch * 32;
    } while (n > 0);
    if (!a.aligned) {
      const float2 p[1] = {make_float2(first, last)};
      add_pairs(r, p, C);
    }
    float m = r.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    // equal maxima keep their sum as it is (infinities included)
    float s = r.m == m ? r.s : r.s * ex2_approx((r.m - m) * a.C);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) a.parts[item.row * a.S + item.part] = make_float2(m, s);
  }
  cp_async_wait<0>();
}

// What the second kernel needs of a row besides its parts.
struct RowInput {
  double w, hit, old_logp, advantage, ref_logp;
};

template <typename T>
__device__ __forceinline__ RowInput row_input(const LossArgs &a, int64_t row) {
  RowInput in = {};
  in.w = a.weight ? (double)a.weight[row] : 1.0 / (double)a.M;
  if (in.w != 0.0) {
    const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
    in.old_logp = (double)a.old_logp[row];
    in.advantage = (double)a.advantage[row];
    if (a.ref_logp) in.ref_logp = (double)a.ref_logp[row];
    // a token outside the vocabulary has no probability: NaN, here and in the loss
    in.hit = tok >= 0 && tok < a.N ? (double)to_f32<T>((static_cast<const T *>(a.z) + row * a.ld)[tok])
                                   : (double)__int_as_float(0x7FC00000);
  }
  return in;
}

// What a row adds to the loss; writes its outputs.
__device__ __forceinline__ double finish_row(const LossArgs &a, int64_t row, const Run &r, const RowInput &in) {
  if (in.w == 0.0) {
    a.logp[row] = 0.0f;
    a.stats[row] = make_float2(0.0f, 0.0f);
    a.coef[row] = 0.0f;
    return 0.0;
  }
  const double s = log((double)r.s);
  const double lp = (in.hit - (double)r.m) * a.inv_t - s;
  const double A = in.advantage;
  const double ratio = exp(lp - in.old_logp);
  const double ra = ratio * A, ca = fmin(fmax(ratio, a.lo), a.hi) * A;
  const bool held = ra > ca;  // the clipped side is the smaller one: no gradient
  double each = held ? -ca : -ra, d = held ? 0.0 : -ra;
  if (a.ref_logp && a.kl != 0.0) {
    const double q = in.ref_logp - lp, em = expm1(q);
    each += a.kl * (em - q);
    d -= a.kl * em;
  }
  a.logp[row] = (float)lp;
  a.stats[row] = make_float2(r.m, (float)s);
  a.coef[row] = (float)(in.w * d);
  return in.w * each;
}

constexpr int kFinishBlock = 128;
constexpr int kThreadParts = 16;  // rows of at most this many parts take a thread each, others a warp

// Joins the rows' parts, finishes the rows and adds the loss: each CTA adds its
// rows in a fixed order, and the CTA that finishes last adds the CTAs' sums in
// order (the count of finished CTAs starts at 0: the first kernel sets it).
// Before the wait for the first kernel a CTA reads its first rows' inputs: that
// kernel lets this one start only after its own wait for what came before, and
// writes none of them.
template <typename T>
__global__ void __launch_bounds__(kFinishBlock) loss_finish_kernel(LossArgs a) {
  __shared__ double sh[kFinishBlock / 32];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31;
  const bool wide = a.S > kThreadParts;
  const int64_t per = wide ? kFinishBlock / 32 : kFinishBlock;  // rows of a CTA step
  int64_t row = blockIdx.x * per + (wide ? tid >> 5 : tid);
  RowInput in = {};
  if (row < a.M) in = row_input<T>(a, row);
  pdl_prologue();
  double sum = 0.0;
  while (row < a.M) {
    Run r;
    if (in.w != 0.0) {
      for (int i = wide ? lane : 0; i < a.S; i += wide ? 32 : 1) {
        const float2 p = a.parts[row * a.S + i];
        Run o;
        o.m = p.x;
        o.s = p.y;
        r = join(r, o, a.C);
      }
    }
    if (wide) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        Run other;
        other.m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o);
        other.s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
        // the lower lane's part first, on both sides: the same bits
        r = (tid & o) ? join(other, r, a.C) : join(r, other, a.C);
      }
    }
    if (!wide || lane == 0) sum += finish_row(a, row, r, in);
    row += per * gridDim.x;
    if (row < a.M) in = row_input<T>(a, row);
  }
  auto cta_sum = [&](double v) {  // to thread 0
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) sh[tid >> 5] = v;
    __syncthreads();
    v = 0.0;
    if (tid == 0)
      for (int w = 0; w < kFinishBlock / 32; ++w) v += sh[w];
    return v;
  };
  sum = cta_sum(sum);
  if (gridDim.x == 1) {
    if (tid == 0) *a.loss = (float)sum;
    return;
  }
  if (tid == 0) {
    a.sums[blockIdx.x] = sum;
    __threadfence();
    last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double s = 0.0;
  for (unsigned i = tid; i < gridDim.x; i += kFinishBlock) s += __ldcg(a.sums + i);
  s = cta_sum(s);
  if (tid == 0) *a.loss = (float)s;
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
