// Log probabilities of given tokens, with the entropy and the best alternatives of
// each row, forward and backward, for sm_100a, from the logits of M rows over a
// vocabulary of N.
//
//   m = max_j z_j,  e_j = (z_j - m) / T,  S = sum_j exp(e_j),  s = log S
//   logp = e_t - s,   entropy = s - sum_j e_j exp(e_j) / S,   top: the K largest logits
//   dz_j = (a ([j = t] - p_j) - b p_j (log p_j + entropy)) / T,   p_j = exp(e_j - s)
//
// The forward is the policy loss's: a warp takes a row or one of S parts of one,
// reads ahead across its items, and keeps a running maximum and the two sums a
// lane. For the alternatives it also leaves the largest logit of every lane's
// batch (a chunk: 8 vectors of 16 bytes), which the running maximum needs
// anyway: one store for 128 bytes read, and no work per element. The K largest
// logits lie in chunks whose largest is at least the K-th largest of the chunks',
// so the second kernel looks for them in a few chunks of the row that it reads again.
//
// Exponents are in binary32 and base 2, as there, and not below -200: 2^-200 is 0
// here, and 0 times an exponent of -inf would be NaN.
#pragma once

#include <type_traits>

#include "dyt_cluster.cuh"
#include "dyt_loss.cuh"

namespace dyt {
namespace loss {

struct LogpArgs {
  const void *z;
  int64_t ld;
  const void *tokens;  // int64 or int32 (wide_tokens); NULL: none, every row counts
  int64_t ignore;      // the token of rows that do not count
  float *logp;         // [M] (with tokens)
  float *entropy;      // [M]
  float2 *stats;       // [M] (m, s)
  float *best;         // [M][K] log probabilities of the largest logits, falling
  long long *ids;      // [M][K] their columns
  float4 *parts;       // [M][most] (maximum, sum of 2^e, sum of e 2^e, -) of each part of a row
  void *tops;          // [M][chunks] of the logits' type, K > 0: each chunk's largest logit
  int *taken;          // the parts that were taken
  int64_t M;
  int64_t N;
  int S;               // parts of a row, unless they are chosen by the list
  int most;            // and how many there is room for
  int batches;         // of kBatch x 32 16-byte vectors in a row, at most
  int listed;          // the first kernel lists the rows that count, and chooses the number of parts for them
  int aligned;         // every row is whole aligned 16-byte vectors
  int wide_tokens;
  int K;
  int together;        // K > 0: rows that a warp of the second kernel takes at a time
  float C;             // log2(e) / T
  double inv_t;
};

struct LogpGradArgs {
  const void *z;
  int64_t ld;
  const void *tokens;  // NULL: none
  int64_t ignore;
  const float2 *stats;
  const float *entropy;  // with db
  const float *da;       // the gradient of logp, NULL: 0
  const float *db;       // the gradient of entropy, NULL: 0
  void *dz;
  int64_t lddz;
  int64_t M;
  int64_t N;
  int S;
  int wide_tokens;
  int lines;
  float C;
  double inv_t;
};

constexpr float kFar = -200.0f;  // the smallest exponent
constexpr double kLn2D = 0.69314718055994530941723212146;

struct Moments {
  float m = kNegInf;  // largest logit so far
  float s = 0.0f;     // sum of 2^e, e = (z - m) C
  float t = 0.0f;     // sum of e 2^e
};

// The sums of r as those about the larger maximum `top`.
__device__ __forceinline__ void raise(Moments &r, float top, float C) {
  if (r.m == top) return;  // (infinities included)
  const float d = max_nan((r.m - top) * C, kFar), f = ex2_approx(d);
  r.t = f * fmaf(d, r.s, r.t);
  r.s *= f;
  r.m = top;
}

__device__ __forceinline__ Moments join(Moments a, Moments b, float C) {
  const float top = fmaxf(a.m, b.m);
  raise(a, top, C);
  raise(b, top, C);
  a.s += b.s;
  a.t += b.t;
  return a;
}

template <typename T>
using Pair = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
template <typename T>
__device__ __forceinline__ Pair<T> half_pair(const uint4 &r, int w) {
  const uint32_t word = word_of(r, w);
  return *reinterpret_cast<const Pair<T> *>(&word);
}
// The largest of 16 bytes of logits, the even and the odd elements apart (x, y); a NaN passes over.
template <typename T>
__device__ __forceinline__ float2 largest(const uint4 &r) {
  if constexpr (sizeof(T) == 4) {
    return make_float2(fmaxf(__uint_as_float(r.x), __uint_as_float(r.z)),
                       fmaxf(__uint_as_float(r.y), __uint_as_float(r.w)));
  } else {
    const Pair<T> m = __hmax2(__hmax2(half_pair<T>(r, 0), half_pair<T>(r, 1)),
                              __hmax2(half_pair<T>(r, 2), half_pair<T>(r, 3)));
    return make_float2(to_f32<T>(m.x), to_f32<T>(m.y));
  }
}
// Pair i of 16 bytes of logits plus c, each rounded once to binary32. (16-bit logits are added as they are.)
template <typename T>
__device__ __forceinline__ float2 plus(const uint4 &r, int i, float c) {
  if constexpr (sizeof(T) == 4) {
    return add2(make_float2(__uint_as_float(word_of(r, 2 * i)), __uint_as_float(word_of(r, 2 * i + 1))), f2(c));
  } else {
    float2 d;
    if constexpr (std::is_same<T, __half>::value)
      asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; add.f32.f16 %0, l, %3; add.f32.f16 %1, h, %3;}"
          : "=f"(d.x), "=f"(d.y)
          : "r"(word_of(r, i)), "f"(c));
    else
      asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; add.f32.bf16 %0, l, %3; add.f32.bf16 %1, h, %3;}"
          : "=f"(d.x), "=f"(d.y)
          : "r"(word_of(r, i)), "f"(c));
    return d;
  }
}

// A whole batch; `top` is its largest logit. NaN passes over the maximum and reaches the sums. Exponents are not looked
// at: the second sum is NaN where one of them was -inf. Nothing is added then, and false returned.
template <typename T>
__device__ __forceinline__ bool add_batch(Moments &r, const uint4 (&raw)[kBatch], float C, float &top) {
  constexpr int P = 8 / (int)sizeof(T);  // pairs of 16 bytes
  if constexpr (sizeof(T) == 4) {
    float x[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      x[0] = max3(x[0], __uint_as_float(raw[u].x), __uint_as_float(raw[u].y));
      x[1] = max3(x[1], __uint_as_float(raw[u].z), __uint_as_float(raw[u].w));
    }
    top = fmaxf(x[0], x[1]);
  } else {
    Pair<T> x[2] = {half_pair<T>(raw[0], 0), half_pair<T>(raw[0], 1)};
#pragma unroll
    for (int i = 2; i < 4 * kBatch; ++i) x[i & 1] = __hmax2(x[i & 1], half_pair<T>(raw[i / 4], i % 4));
    x[0] = __hmax2(x[0], x[1]);
    top = max3(to_f32<T>(x[0].x), to_f32<T>(x[0].y), kNegInf);
  }
  if (top > r.m) raise(r, top, C);
  const float m = r.m == kNegInf ? 0.0f : r.m;  // only -inf so far
  float2 s[2] = {f2(0.0f), f2(0.0f)}, t[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
  for (int u = 0; u < kBatch; ++u)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 e = mul2(plus<T>(raw[u], i, -m), f2(C));
      const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
      s[i & 1] = add2(s[i & 1], p);
      t[i & 1] = fma2(p, e, t[i & 1]);
    }
  s[0] = add2(s[0], s[1]);
  t[0] = add2(t[0], t[1]);
  const float more = t[0].x + t[0].y;
  if (more != more) return false;
  r.s += s[0].x + s[0].y;
  r.t += more;
  return true;
}

// 2 n values more, every exponent kept from -inf; returns the largest.
template <int n>
__device__ __forceinline__ float add_values(Moments &r, const float2 (&v)[n], float C) {
  float x[2] = {fmaxf(v[0].x, v[0].y), kNegInf};
#pragma unroll
  for (int i = 1; i < n; ++i) x[i & 1] = max3(x[i & 1], v[i].x, v[i].y);
  const float top = fmaxf(x[0], x[1]);
  if (top > r.m) raise(r, top, C);
  const float m = r.m == kNegInf ? 0.0f : r.m;  // only -inf so far: every term is 2^-200, which is 0
  float2 s[2] = {f2(0.0f), f2(0.0f)}, t[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float2 e = mul2(add2(v[i], f2(-m)), f2(C));
    e = make_float2(max_nan(e.x, kFar), max_nan(e.y, kFar));
    const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
    s[i & 1] = add2(s[i & 1], p);
    t[i & 1] = fma2(p, e, t[i & 1]);
  }
  s[0] = add2(s[0], s[1]);
  t[0] = add2(t[0], t[1]);
  r.s += s[0].x + s[0].y;
  r.t += t[0].x + t[0].y;
  return top;
}

// The largest of the warp's values; a NaN passes over.
__device__ __forceinline__ float warp_largest(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}

// A warp's sums together, in lane 0: one instruction for the largest, and the two sums by halves of the warp, a lane
// of each half has one.
__device__ __forceinline__ void lanes_together(Moments &r, float C, int lane) {
  raise(r, warp_largest(r.m), C);
  const bool up = (lane & 16) != 0;
  float sum = (up ? r.t : r.s) + __shfl_xor_sync(0xFFFFFFFFu, up ? r.s : r.t, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  r.t = __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
  r.s = sum;
}

// Whether a row counts.
__device__ __forceinline__ bool row_counts(const LogpArgs &a, int64_t row) {
  return a.tokens == nullptr || token_at(a.tokens, a.wide_tokens, row) != a.ignore;
}

// Items, parts, ring and list as in loss_rows_kernel.
// Measured, without alternatives: 8192 x 131072 bf16 349 us (6.15 TB/s; in a long run 360, under the power cap), 4096 x
// 32000 with a quarter of the rows left out 45. Bound by memory and by the exponentials (MUFU 73% busy); short ones by
// their start, the list of rows and the second kernel. An exponential on the FMA pipe by a polynomial costs more in
// issue slots and power than it takes from MUFU; three CTAs an SM spill. With -inf among the logits (masked
// vocabularies: 1% of the columns or 90%, a batch of a warp's has one either way) every batch is computed twice:
// 8192 x 131072 689 us, 4096 x 32000 80.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kRowsBlock, 2) logp_rows_kernel(LogpArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int P = V / 2;
  using IO = VecIO<T, V>;
  extern __shared__ __align__(16) unsigned char dyn[];
  pdl_prologue();
  if (dynamic_smem_bytes() < rows_smem((int)blockDim.x)) return;
  RowList &list = *reinterpret_cast<RowList *>(dyn);  // where the ring will be: done with before the first copy
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4 *ring = reinterpret_cast<uint4 *>(dyn) + warp * (kStages * kBatch * 32) + lane;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t rows = a.M;
  int parts = a.S;
  if (a.listed) {
    rows = list.fill((int)a.M, [&](int row) { return row_counts(a, row) ? 1.0f : 0.0f; });
    parts = choose_parts((float)rows, (float)warps, a.most, a.batches);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.taken = parts;
  const int part_vecs = (a.batches + parts - 1) / parts * (kBatch * 32);
  const float C = a.C;
  int wr = 0, rd = 0;  // the ring's first slots to fill and to read
  // (with a list, every warp of the CTA makes the one step there is)
  for (int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp; a.listed || item < rows * parts;
       item += 32 * warps) {
    const int64_t mine = item + lane * warps;
    int64_t my_row = mine / parts;
    const int my_part = (int)(mine - my_row * parts);
    bool counts = my_row < rows;
    if (counts && a.listed) my_row = list.find((int)my_row, (int)(a.M + 31) / 32);
    else if (counts) counts = row_counts(a, my_row);
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, counts), unread = todo;
    if (a.listed) __syncthreads();  // every warp has looked its items up, all of them
    // Item k's whole vectors: how many, and where they start.
    auto vectors = [&](int k, int64_t &row, int &part, int &head, int &from) {
      row = __shfl_sync(0xFFFFFFFFu, my_row, k);
      part = __shfl_sync(0xFFFFFFFFu, my_part, k);
      head = a.aligned ? 0 : head_elems(static_cast<const T *>(a.z) + row * a.ld, a.N);
      const int nb = (int)((a.N - head) / V);
      // cut at whole batches, so that only a row's last one is not full
      from = min(part * part_vecs, nb);
      return part == parts - 1 ? nb - from : min(part_vecs, nb - from);
    };
    const uint4 *src = nullptr;  // this lane's next vector of the item being read
    int ahead = 0;               // vectors of it not yet asked for
    auto issue = [&]() {
      if (ahead <= 0 && unread) {
        int64_t row;
        int part, head, from;
        ahead = vectors(__ffs((int)unread) - 1, row, part, head, from);
        unread &= unread - 1;
        src = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.z) + row * a.ld + head) + from + lane;
        if (ahead == 0) ahead = 1 - kBatch * 32;  // one batch of nothing
      }
      uint4 *slot = ring + wr;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u * 32 + lane < ahead) cp_async16(slot + u * 32, src + u * 32);
      cp_async_commit();
      src += kBatch * 32;
      ahead -= kBatch * 32;
      wr = wr == (kStages - 1) * kBatch * 32 ? 0 : wr + kBatch * 32;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();
    while (todo) {
      int64_t row;
      int part, head, from;
      int n = vectors(__ffs((int)todo) - 1, row, part, head, from);
      todo &= todo - 1;
      // The elements off the vectors: used only after those, so that nothing waits for them.
      float first = kNegInf, last = kNegInf;
      if (!a.aligned) {
        const T *z = static_cast<const T *>(a.z) + row * a.ld;
        const int tail = (int)((a.N - head) % V);
        if (part == 0 && lane < head) first = to_f32<T>(z[lane]);
        if (part == parts - 1 && lane < tail) last = to_f32<T>(z[a.N - tail + lane]);
      }
      T *tops = nullptr;
      if constexpr (TOP) tops = static_cast<T *>(a.tops) + (row * a.batches + from / (kBatch * 32)) * 32 + lane;
      Moments r;
      do {
        cp_async_wait<kStages - 2>();
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) raw[u] = ring[rd + u * 32];
        const int here = rd;
        rd = rd == (kStages - 1) * kBatch * 32 ? 0 : rd + kBatch * 32;
        issue();
        float top;
        bool done = false;
        if (n >= kBatch * 32) done = add_batch<T>(r, raw, C, top);
        // Batches with infinite exponents (masked logits) are taken once more, and those that end a row at once,
        // a vector at a time with a look at every exponent. Their slots are not filled again before the next batch.
        if (!done) {
          top = kNegInf;
#pragma unroll 1
          for (int u = 0; u * 32 < n && u < kBatch; ++u) {
            float2 v[P];
            IO::unpack2(ring[here + u * 32], v);
            if (u * 32 + lane >= n)
#pragma unroll
              for (int i = 0; i < P; ++i) v[i] = f2(kNegInf);
            top = fmaxf(top, add_values(r, v, C));
          }
        }
        if constexpr (TOP) {
          if (n > 0) *tops = from_f32<T>(top);  // (a part of no vectors has no chunks)
          tops += 32;
        }
        n -= kBatch * 32;
      } while (n > 0);
      if (!a.aligned) {
        const float2 p[1] = {make_float2(first, last)};
        add_values(r, p, C);
      }
      lanes_together(r, C, lane);
      if (lane == 0) a.parts[row * a.most + part] = make_float4(r.m, r.s, r.t, 0.0f);
    }
    // The batches of nothing at the end: the ring starts the next items where it stands.
    cp_async_wait<0>();
    rd = wr;
    if (a.listed) break;
  }
}

// ---- the largest logits ------------------------------------------------------------

// A logit's rank as a whole number: falling logits, rising columns.
using Key = unsigned long long;
__device__ __forceinline__ Key logit_key(float v, uint32_t col) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 is 0
  return (Key)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xFFFFFFFFu - col);
}
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint32_t key_col(Key k) { return 0xFFFFFFFFu - (uint32_t)k; }

constexpr int kMaxTop = DYT_MAX_TOP;  // alternatives, at most: a lane each
static_assert(kMaxTop <= 32, "a lane each");
constexpr int kChunks = 256;  // room for chunks
constexpr int kKeys = 256;    // and for candidates

// A warp's lists, and 8 vectors a lane on their way to it (asynchronous copies: no registers wait for them).
struct __align__(16) Best {
  uint4 stage[8][32];
  Key keys[kKeys];
  Key first[kMaxTop];
  int chunks[kChunks];
};

// A bit for each of 16 bytes of logits that is not below v, a value of T (NaN is).
template <typename T>
__device__ __forceinline__ uint32_t not_below(const uint4 &r, float v) {
  uint32_t m = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) m |= (__uint_as_float(word_of(r, e)) >= v ? 1u : 0u) << e;
  } else {  // pairs: all 16 bits of a half tell
    Pair<T> l;
    l.x = l.y = from_f32<T>(v);
#pragma unroll
    for (int w = 0; w < 4; ++w) m |= __hge2_mask(half_pair<T>(r, w), l) & (0x00020001u << (2 * w));
    m = (m | m >> 16) & 0xFFu;
  }
  return m;
}

// How many elements the lanes before this one have, and all of them.
__device__ __forceinline__ int lanes_before(int count, int lane, int &total) {
  int sum = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += t;
  }
  total = __shfl_sync(0xFFFFFFFFu, sum, 31);
  return sum - count;
}

// The K largest of n keys, in order. (There is room for one more behind them, or n is even.)
__device__ __forceinline__ void rank(Key *keys, int n, Key *out, int K, int lane) {
  if (lane == 0 && (n & 1)) keys[n] = 0;  // they are looked at in pairs; no key is 0
  __syncwarp();
  auto pass = [&](int j, auto pair) {  // a key or two a lane
    constexpr bool two = decltype(pair)::value;
    const Key k0 = j < n ? keys[j] : 0, k1 = two && j + 32 < n ? keys[j + 32] : 0;
    int r0 = 0, r1 = 0;
#pragma unroll 4
    for (int i = 0; i < n; i += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(keys + i);
      r0 += (o.x > k0) + (o.y > k0);
      if (two) r1 += (o.x > k1) + (o.y > k1);
    }
    if (j < n && r0 < K) out[r0] = k0;
    if (two && j + 32 < n && r1 < K) out[r1] = k1;
  };
  int j = lane;
  for (; j - lane + 32 < n; j += 64) pass(j, std::true_type());
  if (j - lane < n) pass(j, std::false_type());
  __syncwarp();
}

// The lanes' values in falling order: lane l gets the l-th largest.
__device__ __forceinline__ float sort_lanes(float v, int lane, int from) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (k < from) continue;
      const float o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
      v = ((lane & j) == 0) == ((lane & k) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// A row's vectors and the largest logits of its chunks. (SHARED: those are in shared memory.)
template <typename T, bool SHARED = false>
struct RowTops {
  static constexpr int V = 16 / (int)sizeof(T);
  const T *z, *tops;
  int head, nb, batches;
  int vecs;  // 16-byte vectors of tops; 0: too few for the warp (less than V batches), taken one by one
  __device__ __forceinline__ RowTops(const LogpArgs &a, int64_t row, const T *all) {
    z = static_cast<const T *>(a.z) + row * a.ld;
    head = a.aligned ? 0 : head_elems(z, a.N);
    nb = (int)((a.N - head) / V);
    batches = (nb + kBatch * 32 - 1) / (kBatch * 32);
    tops = all;
    vecs = batches * 32 / V;
    if (vecs < 32) vecs = 0;
  }
  // The lane's vectors i0 + lane, i0 + lane + 32, ... of tops, 8 of them, into its slots.
  __device__ __forceinline__ void fetch(Best &b, int i0, int lane) const {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u * 32 + lane < vecs)
        if constexpr (SHARED) b.stage[u][lane] = reinterpret_cast<const uint4 *>(tops)[i0 + u * 32 + lane];
        else cp_async16(&b.stage[u][lane], reinterpret_cast<const uint4 *>(tops) + i0 + u * 32 + lane);
    if constexpr (!SHARED) {
      cp_async_commit();
      cp_async_wait<0>();
    }
  }
  // The K-th largest of 64 groups' largest logits, two groups a lane: at least K logits are not below it.
  // Leaves the last 8 vectors of tops in the stage.
  __device__ __forceinline__ float bound(Best &b, int K, int lane) const {
    float2 m = f2(kNegInf);
    if (vecs) {
      for (int i0 = 0; i0 < vecs; i0 += 8 * 32) {
        fetch(b, i0, lane);
#pragma unroll 2
        for (int u = 0; u < 8; ++u) {
          if (i0 + u * 32 + lane >= vecs) break;
          const float2 o = largest<T>(b.stage[u][lane]);
          m = make_float2(fmaxf(m.x, o.x), fmaxf(m.y, o.y));
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < V; u += 2) {
        if (u < batches) m.x = fmaxf(m.x, to_f32<T>(tops[u * 32 + lane]));
        if (u + 1 < batches) m.y = fmaxf(m.y, to_f32<T>(tops[u * 32 + 32 + lane]));
      }
    }
    const float x = sort_lanes(m.x, lane, 0), y = sort_lanes(m.y, lane, 0);
    // the 32 largest of both, in order
    const float v = sort_lanes(fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, y, 31)), lane, 32);
    return __shfl_sync(0xFFFFFFFFu, v, K - 1);
  }
  // Chunk c's first vector.
  __device__ __forceinline__ int first_vec(int c) const { return (c >> 5) * (kBatch * 32) + (c & 31); }
  // The chunk of bit k of a lane's look at 8 vectors of tops from i0 (or at all of few tops, one by one).
  __device__ __forceinline__ int chunk(int i0, int k, int lane) const {
    return vecs ? (i0 + k / V * 32 + lane) * V + k % V : k * 32 + lane;
  }
};

// A bit for each of a lane's 8 vectors of V.
template <int V>
struct Bits {
  using type = typename std::conditional<V == 8, unsigned long long, uint32_t>::type;
  static __device__ __forceinline__ int count(type m) { return V == 8 ? __popcll(m) : __popc((uint32_t)m); }
  static __device__ __forceinline__ int lowest(type m) { return (V == 8 ? __ffsll((long long)m) : __ffs((int)m)) - 1; }
};

// Candidates among the elements off the vectors (less than 32): those not below v.
template <typename T, bool SHARED>
__device__ __forceinline__ int off_vectors(const LogpArgs &a, const RowTops<T, SHARED> &t, float v, Key *keys,
                                           int lane) {
  const int tail = (int)((a.N - t.head) % RowTops<T>::V);
  const bool off = lane < t.head + tail;
  const uint32_t col = lane < t.head ? (uint32_t)lane : (uint32_t)(a.N - tail + lane - t.head);
  const float x = off ? to_f32<T>(t.z[col]) : 0.0f;
  const bool in = off && x >= v;
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
  if (in) keys[__popc(mask & ((1u << lane) - 1u))] = logit_key(x, col);
  return __popc(mask);
}

// The K largest logits of a row into b.first, in order; returns how many there are (K, but for NaN). -1: there
// are more candidates than room, as where many logits are equal.
template <typename T, bool SHARED>
__device__ __forceinline__ int find_best(const LogpArgs &a, const RowTops<T, SHARED> &t, Best &b, int lane) {
  constexpr int V = RowTops<T>::V;
  using B = Bits<V>;
  const int K = a.K;
  const float v = t.bound(b, K, lane);
  int n = off_vectors(a, t, v, b.keys, lane), listed = 0;  // candidates, chunks: the same in every lane
  for (int i0 = 0; i0 == 0 || i0 < t.vecs; i0 += 8 * 32) {
    typename B::type mask = 0;
    if (t.vecs > 8 * 32) t.fetch(b, i0, lane);
    if (t.vecs) {
#pragma unroll 2
      for (int u = 0; u < 8; ++u) {
        if (i0 + u * 32 + lane >= t.vecs) break;
        mask |= (typename B::type)not_below<T>(b.stage[u][lane], v) << (u * V);
      }
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (u < t.batches) mask |= (typename B::type)(to_f32<T>(t.tops[u * 32 + lane]) >= v) << u;
    }
    int total, at = lanes_before(B::count(mask), lane, total);
    if (listed + total > kChunks) return -1;
    for (at += listed; mask; mask &= mask - 1) b.chunks[at++] = t.chunk(i0, B::lowest(mask), lane);
    listed += total;
  }
  __syncwarp();
  const uint4 *zv = reinterpret_cast<const uint4 *>(t.z + t.head);
  for (int i = lane; i - lane < listed; i += 32) {  // a chunk a lane
    const int first = i < listed ? t.first_vec(b.chunks[i]) : t.nb;
    const int vecs = min(kBatch, (t.nb - first + 31) / 32);  // of the chunk
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (u < vecs) cp_async16(&b.stage[u][lane], zv + first + u * 32);
    cp_async_commit();
    cp_async_wait<0>();
    typename B::type mask = 0;
#pragma unroll 2
    for (int u = 0; u < vecs; ++u) mask |= (typename B::type)not_below<T>(b.stage[u][lane], v) << (u * V);
    int total, at = lanes_before(B::count(mask), lane, total);
    if (n + total > kKeys) return -1;
    for (at += n; mask; mask &= mask - 1) {
      const int k = B::lowest(mask);
      b.keys[at++] = logit_key(to_f32<T>(reinterpret_cast<const T *>(&b.stage[k / V][lane])[k % V]),
                               (uint32_t)(t.head + (first + k / V * 32) * V + k % V));
    }
    n += total;
  }
  rank(b.keys, n, b.first, K, lane);
  return min(n, K);
}

// The same where candidates are many: a chunk at a time, all but the K largest dropped whenever there is no room.
template <typename T, bool SHARED>
__device__ __noinline__ int find_best_of_many(const LogpArgs &a, int64_t row, const T *tops, Best &b, int lane) {
  constexpr int V = RowTops<T>::V;
  const RowTops<T, SHARED> t(a, row, tops);
  const int K = a.K;
  Key least = logit_key(t.bound(b, K, lane), 0xFFFFFFFFu);  // of that value at any column
  __syncwarp();
  int n = off_vectors(a, t, key_value(least), b.keys, lane);
  auto prune = [&]() {
    rank(b.keys, n, b.first, K, lane);
    if (n >= K) least = b.first[K - 1];
    n = min(n, K);
    if (lane < n) b.keys[lane] = b.first[lane];
    __syncwarp();
  };
  for (int c0 = 0; c0 < t.batches * 32; c0 += 32) {
    // a chunk's logits stand behind its first one
    const int first = t.first_vec(c0 + lane);
    const bool could = logit_key(to_f32<T>(t.tops[c0 + lane]), (uint32_t)(t.head + first * V)) >= least;
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, could);
    while (todo) {
      const int c = c0 + __ffs((int)todo) - 1;
      todo &= todo - 1;
      for (int o = lane; o - lane < kBatch * V; o += 32) {  // its logits, 32 at a time
        const int vec = t.first_vec(c) + o / V * 32, e = vec * V + o % V;
        const bool in = vec < t.nb;
        const float x = in ? to_f32<T>(t.z[t.head + e]) : 0.0f;
        const Key k = logit_key(x, (uint32_t)(t.head + e));
        const bool take = in && x == x && k >= least;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, take);
        if (take) b.keys[n + __popc(mask & ((1u << lane) - 1u))] = k;
        n += __popc(mask);
        if (n > kKeys / 2) prune();
      }
    }
  }
  prune();
  return n;
}

// ---- second kernel -----------------------------------------------------------------

// What is read of a row before the first kernel is waited for (see loss_finish_kernel: this one too is launched
// directly after its first kernel, and that one releases it nowhere but in pdl_prologue).
struct LogpInput {
  bool counts = false;
  double hit = 0.0;
};
template <typename T>
__device__ __forceinline__ LogpInput logp_input(const LogpArgs &a, int64_t row) {
  LogpInput in;
  in.counts = true;
  if (a.tokens) {
    const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
    in.counts = tok != a.ignore;
    // a token outside the vocabulary has no probability
    in.hit = (double)__int_as_float(0x7FC00000);
    if (in.counts && tok >= 0 && tok < a.N)
      in.hit = (double)to_f32<T>(__ldcg(static_cast<const T *>(a.z) + row * a.ld + tok));
  }
  return in;
}

// Parts first, first + step, ... of a row.
__device__ __forceinline__ Moments some_parts(const LogpArgs &a, int64_t row, int parts, int first, int step) {
  Moments r;
  for (int i = first; i < parts; i += step) {
    const float4 p = a.parts[row * a.most + i];
    Moments o;
    o.m = p.x;
    o.s = p.y;
    o.t = p.z;
    r = join(r, o, a.C);
  }
  return r;
}
// The lanes' parts together.
__device__ __forceinline__ Moments join_lanes(Moments r, float C) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Moments other;
    other.m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o);
    other.s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
    other.t = __shfl_xor_sync(0xFFFFFFFFu, r.t, o);
    // the lower lane's part first, on both sides: the same bits
    r = (threadIdx.x & o) ? join(other, r, C) : join(r, other, C);
  }
  return r;
}
// Writes a row's outputs; returns the log of its sum.
__device__ __forceinline__ double finish_row(const LogpArgs &a, int64_t row, const Moments &r, const LogpInput &in) {
  if (!in.counts) {
    if (a.logp) a.logp[row] = 0.0f;
    a.entropy[row] = 0.0f;
    a.stats[row] = make_float2(0.0f, 0.0f);
    return 0.0;
  }
  const double s = log((double)r.s);
  if (a.logp) a.logp[row] = (float)((in.hit - (double)r.m) * a.inv_t - s);
  a.entropy[row] = (float)(s - kLn2D * ((double)r.t / (double)r.s));
  a.stats[row] = make_float2(r.m, (float)s);
  return s;
}

// Joins the rows' parts and finishes the rows: a thread each, or a warp where there are many parts.
template <typename T>
__global__ void __launch_bounds__(kFinishBlock) logp_finish_kernel(LogpArgs a) {
  const int tid = threadIdx.x, lane = tid & 31;
  const bool wide = a.most > kThreadParts;
  const int64_t per = wide ? kFinishBlock / 32 : kFinishBlock;  // rows of a CTA step
  int64_t row = blockIdx.x * per + (wide ? tid >> 5 : tid);
  LogpInput in;
  if (row < a.M) in = logp_input<T>(a, row);
  pdl_prologue();
  const int parts = *a.taken;
  while (row < a.M) {
    Moments r;
    if (in.counts) r = some_parts(a, row, parts, wide ? lane : 0, wide ? 32 : 1);
    if (wide) r = join_lanes(r, a.C);
    if (!wide || lane == 0) finish_row(a, row, r, in);
    row += per * gridDim.x;
    if (row < a.M) in = logp_input<T>(a, row);
  }
}

// A row's alternatives, from its maximum and the log of its sum.
template <typename T, bool SHARED>
__device__ __forceinline__ void write_best(const LogpArgs &a, int64_t row, const T *tops, bool counts, double m,
                                           double s, Best &b, int lane) {
  int n = 0;
  if (counts) {
    n = find_best<T>(a, RowTops<T, SHARED>(a, row, tops), b, lane);
    if (n < 0) n = find_best_of_many<T, SHARED>(a, row, tops, b, lane);
  }
  if (lane < a.K) {
    const bool found = lane < n;
    const Key key = found ? b.first[lane] : 0;
    const float none = counts ? __int_as_float(0x7FC00000) : 0.0f;
    const int64_t at = row * a.K + lane;
    a.best[at] = found ? (float)(((double)key_value(key) - m) * a.inv_t - s) : none;
    a.ids[at] = found ? (long long)key_col(key) : -1;
  }
}

constexpr int kTopBlock = 128, kTopCtas = 6;  // CTAs that an SM holds
// The same with alternatives. A warp takes `a.together` rows at a time: a lane each for their parts and their scalars,
// all lanes for each row's alternatives. (One row: all lanes for its parts too.)
// Measured, both kernels: 8192 x 131072 bf16 without alternatives 349 us, with 8 of them 388, with 20 406, with 32 432
// (4 KB of chunk maxima a row are written and read, and a few chunks read again). Bound by latency: a row is four trips
// to memory one after the other (maxima, chunks over the bound, their logits, outputs), with 24 warps an SM to hide
// them.
template <typename T>
__global__ void __launch_bounds__(kTopBlock, kTopCtas) logp_top_kernel(const __grid_constant__ LogpArgs a) {
  __shared__ Best best[kTopBlock / 32];
  const int lane = threadIdx.x & 31;
  Best &b = best[threadIdx.x >> 5];
  const int R = a.together;
  const int64_t step = (int64_t)gridDim.x * (kTopBlock / 32) * R;
  int64_t base = ((int64_t)blockIdx.x * (kTopBlock / 32) + (threadIdx.x >> 5)) * R;
  LogpInput in;
  if (lane < R && base + lane < a.M) in = logp_input<T>(a, base + lane);
  pdl_prologue();
  const int parts = *a.taken;
  while (base < a.M) {
    const int rows = (int)min((int64_t)R, a.M - base);
    Moments mine;
    double s = 0.0;
    if (R == 1) {
      in.counts = __shfl_sync(0xFFFFFFFFu, in.counts, 0);
      if (in.counts) mine = some_parts(a, base, parts, lane, 32);
      mine = join_lanes(mine, a.C);
    } else if (in.counts) {
      mine = some_parts(a, base + lane, parts, 0, 1);
    }
    if (lane < rows) s = finish_row(a, base + lane, mine, in);
    const uint32_t counting = __ballot_sync(0xFFFFFFFFu, in.counts && lane < rows);
    for (int k = 0; k < rows; ++k) {
      const bool counts = counting >> k & 1u;
      const double m_k = (double)__shfl_sync(0xFFFFFFFFu, mine.m, k), s_k = __shfl_sync(0xFFFFFFFFu, s, k);
      const T *tops = static_cast<const T *>(a.tops) + (base + k) * a.batches * 32;
      write_best<T, false>(a, base + k, tops, counts, m_k, s_k, b, lane);
      __syncwarp();  // (the next row's candidates take their place)
    }
    base += step;
    in = LogpInput();
    if (lane < R && base + lane < a.M) in = logp_input<T>(a, base + lane);
  }
}

// ---- few rows ---------------------------------------------------------------------------

constexpr int kFewWarps = 8;       // of a CTA
constexpr int kFewBatches = 256;   // of a row, at most (2 x 500000 binary32, 489: 30.5 us, in two kernels 29.1)

// A row is a cluster's (dyt_cluster.cuh), a batch at a time a warp's; its sums and its chunks' largest logits meet in
// the first CTA's shared memory, whose first warp finishes the row: one launch, and no workspace. Measured: 1 x 131072
// bf16 4.4 us, with 20 alternatives 8.2; 7 x 50001 binary32 with 20 10.3. Bound by latency: the batch, the exchange,
// the chunks over the bound and the ranking one after the other.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kFewWarps * 32) logp_few_kernel(const __grid_constant__ LogpArgs a) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2;
  using IO = VecIO<T, V>;
  __shared__ float4 parts[kMaxCluster * kFewWarps];
  __shared__ Best best;
  extern __shared__ __align__(16) unsigned char dyn[];
  pdl_prologue();
  if (TOP && dynamic_smem_bytes() < (size_t)a.batches * 32 * sizeof(T)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_ctas();
  const int64_t row = blockIdx.x / ctas;
  T *const tops = reinterpret_cast<T *>(dyn);
  const float C = a.C;
  const bool counts = row_counts(a, row);  // (all of the cluster agree)
  LogpInput in;
  if (rank == 0 && threadIdx.x == 0) in = logp_input<T>(a, row);
  Moments r;
  if (counts) {
    const RowTops<T, true> t(a, row, tops);
    const uint4 *zv = reinterpret_cast<const uint4 *>(t.z + t.head);
    cluster_sync();  // all CTAs have started
    for (int b = (int)rank * warps + warp; b < t.batches; b += (int)ctas * warps) {
      const uint4 *src = zv + b * (kBatch * 32) + lane;
      const int n = t.nb - b * (kBatch * 32);
      float top;
      bool done = false;
      if (n >= kBatch * 32) {
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) raw[u] = __ldcg(src + u * 32);
        done = add_batch<T>(r, raw, C, top);
      }
      if (!done) {  // (see logp_rows_kernel)
        top = kNegInf;
#pragma unroll 1
        for (int u = 0; u * 32 < n && u < kBatch; ++u) {
          float2 v[P];
#pragma unroll
          for (int i = 0; i < P; ++i) v[i] = f2(kNegInf);
          if (u * 32 + lane < n) IO::unpack2(__ldcg(src + u * 32), v);
          top = fmaxf(top, add_values(r, v, C));
        }
      }
      if constexpr (TOP) cluster_put(tops + b * 32 + lane, 0u, from_f32<T>(top));
    }
    if (!a.aligned && rank == 0 && warp == 0) {  // the elements off the vectors
      const int tail = (int)((a.N - t.head) % V);
      const float2 p[1] = {make_float2(lane < t.head ? to_f32<T>(t.z[lane]) : kNegInf,
                                       lane < tail ? to_f32<T>(t.z[a.N - tail + lane]) : kNegInf)};
      add_values(r, p, C);
    }
    lanes_together(r, C, lane);
    if (lane == 0) cluster_put(parts + rank * warps + warp, 0u, make_float4(r.m, r.s, r.t, 0.0f));
    cluster_sync();
  }
  if (rank != 0 || warp != 0) return;
  Moments mine;
  if (counts) {
    for (int i = lane; i < (int)ctas * warps; i += 32) {
      const float4 p = parts[i];
      Moments o;
      o.m = p.x;
      o.s = p.y;
      o.t = p.z;
      mine = join(mine, o, C);
    }
    mine = join_lanes(mine, C);
  }
  double s = 0.0;
  if (lane == 0) s = finish_row(a, row, mine, in);
  if constexpr (TOP)
    write_best<T, true>(a, row, tops, counts, (double)__shfl_sync(0xFFFFFFFFu, mine.m, 0),
                        __shfl_sync(0xFFFFFFFFu, s, 0), best, lane);
}

// ---- backward -------------------------------------------------------------------------

// The gradient in a row: A [j = tok] + (c0 + c1 e) 2^e, e = (z - m) C, with p = 2^e e^-s and
// log p + entropy = e ln 2 - s + entropy.
// Measured in loss_grad_kernel: 8192 x 131072 bf16 635 us (6.76 TB/s), 16384 x 4096 bf16 44 (6.1), 4096 x 32003 fp16
// with a quarter of the rows left out 77 (5.9). Bound by memory.
struct LogpGradRow {
  using Args = LogpGradArgs;
  struct Call {
    __device__ __forceinline__ Call(const Args &) {}
  };
  int64_t tok;
  float A, c0, c1, m, C;
  bool none;
  __device__ __forceinline__ LogpGradRow(const Args &a, const Call &, int64_t row) : C(a.C) {
    float da = a.da ? a.da[row] : 0.0f;
    float db = a.db ? a.db[row] : 0.0f;
    const float h = a.db ? a.entropy[row] : 0.0f;
    const float2 st = a.stats[row];
    tok = a.tokens ? token_at(a.tokens, a.wide_tokens, row) : -1;
    if (a.tokens && tok == a.ignore) da = db = 0.0f;
    none = da == 0.0f && db == 0.0f;
    m = st.x;
    const float q = expf(-st.y), b = (float)((double)db * a.inv_t);
    A = (float)((double)da * a.inv_t);
    c0 = -q * (A + b * (h - st.y));
    c1 = -q * (b * (float)kLn2D);
    // the token has no probability: neither has the row a gradient
    if (da != 0.0f && (tok < 0 || tok >= a.N)) c0 = __int_as_float(0x7FC00000);
  }
  __device__ __forceinline__ bool zero() const { return none; }
  __device__ __forceinline__ float2 pair(float2 z) const {
    float2 e = mul2(add2(z, f2(-m)), f2(C));
    e = make_float2(max_nan(e.x, kFar), max_nan(e.y, kFar));
    return mul2(make_float2(ex2_approx(e.x), ex2_approx(e.y)), fma2(f2(c1), e, f2(c0)));
  }
};

}  // namespace loss
}  // namespace dyt
