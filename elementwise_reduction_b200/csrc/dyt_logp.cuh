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

// 2 n values more; returns the largest. NaN passes over the maximum and reaches the sums.
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

// Whether a row counts.
__device__ __forceinline__ bool row_counts(const LogpArgs &a, int64_t row) {
  return a.tokens == nullptr || token_at(a.tokens, a.wide_tokens, row) != a.ignore;
}

// Items, parts, ring and list as in loss_rows_kernel.
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
        rd = rd == (kStages - 1) * kBatch * 32 ? 0 : rd + kBatch * 32;
        issue();
        float2 v[kBatch * P];
        float top;
        if (n >= kBatch * 32) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) IO::unpack2(raw[u], *reinterpret_cast<float2(*)[P]>(v + u * P));
          top = add_values(r, v, C);
        } else {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            IO::unpack2(raw[u], *reinterpret_cast<float2(*)[P]>(v + u * P));
            if (u * 32 + lane >= n)
#pragma unroll
              for (int i = 0; i < P; ++i) v[u * P + i] = f2(kNegInf);
          }
          top = add_values(r, v, C);
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
      float m = r.m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      raise(r, m, C);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
        r.t += __shfl_xor_sync(0xFFFFFFFFu, r.t, o);
      }
      if (lane == 0) a.parts[row * a.most + part] = make_float4(r.m, r.s, r.t, 0.0f);
    }
    // The batches of nothing at the end: the ring starts the next items where it stands.
    cp_async_wait<0>();
    rd = wr;
    if (a.listed) break;
  }
}

// ---- the largest logits ------------------------------------------------------------

// A logit's rank as a whole number: falling logits, rising columns. 0: none.
using Key = unsigned long long;
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ Key logit_key(float v, uint32_t col) { return (Key)value_key(v) << 32 | (0xFFFFFFFFu - col); }
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint32_t key_col(Key k) { return 0xFFFFFFFFu - (uint32_t)k; }

constexpr int kMaxTop = DYT_MAX_TOP;  // alternatives, at most: a lane each
static_assert(kMaxTop <= 32, "a lane each");
constexpr int kChunks = 256;  // chunks listed before they are read
constexpr int kKeys = 256;    // candidates kept before all but K of them are dropped

// A warp's candidates: every logit not below `least`, which rises to the K-th largest seen.
struct Best {
  Key keys[kKeys];
  int chunks[kChunks];
};
struct BestState {
  Key least;
  int n;  // candidates
};

// All but the K largest candidates go; those stand in order.
__device__ __forceinline__ void prune(Best &b, BestState &st, int K, int lane) {
  __syncwarp();
  Key mine[kKeys / 32];
  int rank[kKeys / 32];
#pragma unroll
  for (int j = 0; j < kKeys / 32; ++j) {
    mine[j] = j * 32 + lane < st.n ? b.keys[j * 32 + lane] : 0;
    rank[j] = 0;
  }
  for (int i = 0; i < st.n; ++i) {
    const Key k = b.keys[i];
#pragma unroll
    for (int j = 0; j < kKeys / 32; ++j)
      if (j * 32 < st.n) rank[j] += k > mine[j];
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kKeys / 32; ++j)
    if (j * 32 + lane < st.n && rank[j] < K) b.keys[rank[j]] = mine[j];
  st.n = min(st.n, K);
  __syncwarp();
  if (st.n == K) st.least = b.keys[K - 1];
}

__device__ __forceinline__ void push(Best &b, BestState &st, bool in, float v, uint32_t col, int K, int lane) {
  const Key k = logit_key(v, col);
  in = in && v == v && k >= st.least;  // NaN is no alternative
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
  if (mask == 0) return;
  if (in) b.keys[st.n + __popc(mask & ((1u << lane) - 1u))] = k;
  st.n += __popc(mask);
  if (st.n > kKeys - 32) prune(b, st, K, lane);
}

// The K largest logits of a row into b.keys[0 .. st.n).
template <typename T>
__device__ __forceinline__ void find_best(const LogpArgs &a, int64_t row, Best &b, BestState &st, int lane) {
  constexpr int V = 16 / (int)sizeof(T);
  const int K = a.K;
  const T *z = static_cast<const T *>(a.z) + row * a.ld;
  const int head = a.aligned ? 0 : head_elems(z, a.N);
  const int nb = (int)((a.N - head) / V), tail = (int)((a.N - head) % V);
  const int batches = (nb + kBatch * 32 - 1) / (kBatch * 32);
  const T *tops = static_cast<const T *>(a.tops) + row * a.batches * 32 + lane;
  // The K-th largest of the lanes' largest chunks: at least K logits are not below it.
  float mine = kNegInf;
#pragma unroll 8
  for (int i = 0; i < batches; ++i) mine = fmaxf(mine, to_f32<T>(tops[i * 32]));
  const uint32_t o = value_key(mine);
  int above = 0;
#pragma unroll
  for (int l = 0; l < 32; ++l) {
    const uint32_t other = __shfl_sync(0xFFFFFFFFu, o, l);
    above += other > o || (other == o && l < lane);
  }
  const uint32_t kth = __ballot_sync(0xFFFFFFFFu, above == K - 1);
  st.least = (Key)__shfl_sync(0xFFFFFFFFu, o, __ffs((int)kth) - 1) << 32;
  st.n = 0;
  if (head > 0) push(b, st, lane < head, lane < head ? to_f32<T>(z[lane]) : 0.0f, (uint32_t)lane, K, lane);
  if (tail > 0)
    push(b, st, lane < tail, lane < tail ? to_f32<T>(z[a.N - tail + lane]) : 0.0f, (uint32_t)(a.N - tail + lane), K,
         lane);
  int listed = 0;
  // A chunk is kBatch vectors: a lane takes four bytes of one, several chunks under way at once.
  auto read_chunks = [&]() {
    __syncwarp();
    constexpr int U = 4, W = 4 / (int)sizeof(T);
    for (int i = 0; i < listed; i += U) {
      uint32_t raw[U], col[U];
      bool in[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = i + u < listed ? b.chunks[i + u] : 0;
        const int vec = (c >> 5) * (kBatch * 32) + (lane >> 2) * 32 + (c & 31);
        in[u] = i + u < listed && vec < nb;
        col[u] = (uint32_t)(head + vec * V + (lane & 3) * W);
        raw[u] = in[u] ? *reinterpret_cast<const uint32_t *>(z + col[u]) : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (sizeof(T) == 4) {
          push(b, st, in[u], __uint_as_float(raw[u]), col[u], K, lane);
        } else {
          const T *h = reinterpret_cast<const T *>(&raw[u]);
          push(b, st, in[u], to_f32<T>(h[0]), col[u], K, lane);
          push(b, st, in[u], to_f32<T>(h[1]), col[u] + 1, K, lane);
        }
      }
    }
    listed = 0;
    __syncwarp();
  };
  constexpr int B = 4;  // batches looked at together
  for (int i0 = 0; i0 < batches; i0 += B) {
    float top[B];
#pragma unroll
    for (int u = 0; u < B; ++u) top[u] = i0 + u < batches ? to_f32<T>(tops[(i0 + u) * 32]) : kNegInf;
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int vec = (i0 + u) * (kBatch * 32) + lane;
      // the chunk's best key, if its largest logit stood first
      const bool in = vec < nb && logit_key(top[u], (uint32_t)(head + vec * V)) >= st.least;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
      if (in) b.chunks[listed + __popc(mask & ((1u << lane) - 1u))] = (i0 + u) * 32 + lane;
      listed += __popc(mask);
    }
    if (listed > kChunks - 32 * B) read_chunks();
  }
  read_chunks();
  prune(b, st, K, lane);
}

// ---- second kernel -----------------------------------------------------------------

constexpr int kTopCtasPerSm = 8;

// Joins the rows' parts and finishes the rows. A row takes a thread, or a warp (with alternatives, or of
// many parts). As in loss_finish_kernel, a CTA reads its first rows' tokens and their logits before the wait.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kFinishBlock) logp_finish_kernel(LogpArgs a) {
  __shared__ Best best[TOP ? kFinishBlock / 32 : 1];
  const int tid = threadIdx.x, lane = tid & 31;
  const bool wide = TOP || a.most > kThreadParts;
  const int64_t per = wide ? kFinishBlock / 32 : kFinishBlock;  // rows of a CTA step
  struct Input {
    bool counts;
    double hit;
  };
  auto input = [&](int64_t row) {
    Input in = {true, 0.0};
    if (a.tokens) {
      const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
      in.counts = tok != a.ignore;
      // a token outside the vocabulary has no probability
      in.hit = (double)__int_as_float(0x7FC00000);
      if (in.counts && tok >= 0 && tok < a.N)
        in.hit = (double)to_f32<T>(__ldcg(static_cast<const T *>(a.z) + row * a.ld + tok));
    }
    return in;
  };
  int64_t row = blockIdx.x * per + (wide ? tid >> 5 : tid);
  Input in = {};
  if (row < a.M) in = input(row);
  pdl_prologue();
  const int parts = *a.taken;
  while (row < a.M) {
    Moments r;
    if (in.counts) {
      for (int i = wide ? lane : 0; i < parts; i += wide ? 32 : 1) {
        const float4 p = a.parts[row * a.most + i];
        Moments o;
        o.m = p.x;
        o.s = p.y;
        o.t = p.z;
        r = join(r, o, a.C);
      }
    }
    if (wide) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        Moments other;
        other.m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o);
        other.s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
        other.t = __shfl_xor_sync(0xFFFFFFFFu, r.t, o);
        // the lower lane's part first, on both sides: the same bits
        r = (tid & o) ? join(other, r, a.C) : join(r, other, a.C);
      }
    }
    const double s = in.counts ? log((double)r.s) : 0.0;
    if (!wide || lane == 0) {
      if (a.logp) a.logp[row] = in.counts ? (float)((in.hit - (double)r.m) * a.inv_t - s) : 0.0f;
      a.entropy[row] = in.counts ? (float)(s - kLn2D * ((double)r.t / (double)r.s)) : 0.0f;
      a.stats[row] = in.counts ? make_float2(r.m, (float)s) : make_float2(0.0f, 0.0f);
    }
    if constexpr (TOP) {
      Best &b = best[tid >> 5];
      BestState st = {0, 0};
      if (in.counts) find_best<T>(a, row, b, st, lane);
      if (lane < a.K) {
        const bool found = lane < st.n;
        const Key k = found ? b.keys[lane] : 0;
        const float none = in.counts ? __int_as_float(0x7FC00000) : 0.0f;
        a.best[row * a.K + lane] = found ? (float)(((double)key_value(k) - (double)r.m) * a.inv_t - s) : none;
        a.ids[row * a.K + lane] = found ? (long long)key_col(k) : -1;
      }
      __syncwarp();  // (the next row's candidates take their place)
    }
    row += per * gridDim.x;
    if (row < a.M) in = input(row);
  }
}

// ---- backward -------------------------------------------------------------------------

// The gradient in a row: A [j = tok] + (c0 + c1 e) 2^e, e = (z - m) C, with p = 2^e e^-s and
// log p + entropy = e ln 2 - s + entropy.
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
