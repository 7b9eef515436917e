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
// C's rounding (up to 2^-24, the same way in every term) puts a row's log sum off by
// that share of the mean of |z - m| / T under the row's probabilities. Measured over 512
// rows at T = 0.7, where it is near its largest: log probabilities 3.3e-7 off on average
// (131072 bf16; half of that is their own rounding, and the plain binary32 form's
// 4.2e-7), with the constant in two parts 3.1e-7, for 3 to 4% more time.
#pragma once

#include "dyt_async.cuh"

namespace dyt {
namespace loss {

constexpr float kNegInf = -__builtin_huge_valf();
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
  float2 *parts;           // [M][most] (maximum, sum of 2^((z - maximum) C)) of each part of a row
  double *sums;            // [CTA of the second kernel] what its rows add to the loss
  unsigned *done;          // how many of those CTAs have finished; the parts that were taken
  int64_t M;
  int64_t N;
  int S;                   // parts of a row, unless they are chosen by the list
  int most;                // and how many there is room for
  int batches;             // of kBatch x 32 16-byte vectors in a row, at most
  int listed;              // the first kernel lists the rows that count, and chooses the number of parts for them
  int aligned;             // every row is whole aligned 16-byte vectors
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
  int lines;          // every row is whole 128-byte lines: they are not needed again
  float C;
  double inv_t;
};

__device__ __forceinline__ int64_t token_at(const void *p, int wide, int64_t row) {
  return wide ? __ldcg(static_cast<const long long *>(p) + row) : (int64_t)__ldcg(static_cast<const int *>(p) + row);
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

__host__ __device__ constexpr size_t rows_smem(int block) { return (size_t)block * kBatch * kStages * 16; }

// The parts of a row of `batches` batches, at most `most`: two items for every
// warp if that leaves a part of a long row three batches (the next item's copies then run under
// the current one's end), and a few more where that makes the warps' rounds more
// nearly whole; else one round of items, as many as there are warps. Measured,
// us, bf16 over 2368 warps: 4096 rows of 32000 (16 batches), 1.73 rounds whole,
// 58.4, 6.92 in four parts, 48.9, 13.8 in eight 51.5; 2000 rows of 131072 in five 87.7,
// ten 91.6; 400 rows of 50000 in five parts, one round, 14.9, in eight 17.4, in twelve 17.8.
constexpr int kListedParts = 16;  // room for at least so many (or all of a row's batches), where the kernel chooses
constexpr int kPartBatches = 3;   // at least, in more than one round
__host__ __device__ inline int choose_parts(float rows, float warps, int most, int batches) {
  const float least = ceilf(2.0f * warps / fmaxf(rows, 1.0f));
  // (short rows: down to a batch)
  int cap = batches < 2 * kPartBatches ? batches : (batches + kPartBatches - 1) / kPartBatches;
  if (cap > most) cap = most;
  if (least > (float)cap) {
    const float one = floorf(warps / fmaxf(rows, 1.0f));
    return one < 1.0f ? 1 : one < (float)most ? (int)one : most;
  }
  int S = (int)least;
  if (S < 1) S = 1;
  float best = 0.0f;
  int chosen = S;
  for (int last = S + 8 < cap ? S + 8 : cap; S <= last; ++S) {
    const float rounds = rows * (float)S / warps, even = rounds / ceilf(rounds);
    if (even > best + 0.02f) {
      best = even;
      chosen = S;
    }
  }
  return chosen;
}

// Which of the first kMaxListed rows count: a bit each, and how many do before
// each word of bits. Every CTA makes the list itself, so that warps take equal
// numbers of rows that count however the weights lie. A warp looks up at most 32
// items, so the rows times the parts that there is room for must not pass that
// many a warp: on 148 SMs 8192 rows of less than 10 batches, 4736 of 16 and more
// (vocabularies of 32768 in 16 bits). Beyond it weights are looked up item by item.
constexpr int kMaxListed = 8192;
struct RowList {
  uint32_t bits[kMaxListed / 32];
  int before[kMaxListed / 32 + 1];

  // All kRowsBlock threads of the CTA; returns how many rows count.
  __device__ __forceinline__ int fill(const LossArgs &a) {
    const int M = (int)a.M, words = (M + 31) / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kRowsBlock / 32, kAtOnce = 16;  // the weights of so many words are under way together
    for (int w0 = warp; w0 < words; w0 += kAtOnce * kWarps) {
      float v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int row = (w0 + i * kWarps) * 32 + lane;
        v[i] = row < M ? a.weight[row] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, v[i] != 0.0f);
        if (lane == 0 && w0 + i * kWarps < words) bits[w0 + i * kWarps] = b;
      }
    }
    __syncthreads();
    if (warp == 0) {
      int base = 0;
      for (int w0 = 0; w0 < words; w0 += 32) {
        const int n = w0 + lane < words ? __popc(bits[w0 + lane]) : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += t;
        }
        if (w0 + lane < words) before[w0 + lane] = base + sum - n;
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
      if (lane == 0) before[words] = base;
    }
    __syncthreads();
    return before[words];
  }
  // The row of that rank among those that count.
  __device__ __forceinline__ int find(int rank, int words) const {
    int lo = 0, hi = words;  // before[lo] <= rank < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= rank) lo = mid;
      else hi = mid;
    }
    uint32_t b = bits[lo];
    int n = rank - before[lo], at = 0;  // the n-th set bit
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const int c = __popc(b & ((1u << s) - 1u));
      if (n >= c) {
        n -= c;
        b >>= s;
        at += s;
      }
    }
    return lo * 32 + at;
  }
};

// The items are (row, part), a row's parts one after the other, rows of weight
// 0 left out. A warp takes items w, w + warps, ..., 32 at a time:
// lane k looks up the k-th one, then the warp reads them one after the other.
// A row's whole 16-byte vectors are cut into parts, the elements before and
// after them go with the first and the last part. Every lane keeps kStages
// batches of vectors in a ring of its own (asynchronous copies), across items.
// Measured, with the second kernel: 16384 x 131072 bf16 648 us (6.6 TB/s; under
// the power cap 710), 4096 x 32000 with a quarter of the rows without weight 43
// us, 7 x 50001 fp32 6.6 us. Bound by memory, and by the exponentials (one MUFU
// instruction an element: 77% of that unit's rate) when the clock falls. A CTA
// per row without reading ahead took 47 us for 4096 x 32000, a part-by-part
// order of the items (neighbouring warps in different rows) 46.
template <typename T>
__global__ void __launch_bounds__(kRowsBlock, 2) loss_rows_kernel(LossArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int P = V / 2;
  using IO = VecIO<T, V>;
  extern __shared__ __align__(16) unsigned char dyn[];
  pdl_prologue();
  if (dynamic_smem_bytes() < rows_smem((int)blockDim.x)) return;
  // The list lies where the ring will: it is done with before the first copy.
  // (2 KB more shared memory leave the SM 28 KB of L1 instead of 60, and the
  // pass over 16384 x 131072 bf16 takes 742 us instead of 642.)
  RowList &list = *reinterpret_cast<RowList *>(dyn);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4 *ring = reinterpret_cast<uint4 *>(dyn) + warp * (kStages * kBatch * 32) + lane;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t rows = a.M;
  int parts = a.S;
  if (a.listed) {
    rows = list.fill(a);
    parts = choose_parts((float)rows, (float)warps, a.most, a.batches);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.done[0] = 0u;
    a.done[1] = (unsigned)parts;
  }
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
    else if (counts && a.weight) counts = a.weight[my_row] != 0.0f;
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, counts), unread = todo;
    if (a.listed) __syncthreads();  // every warp has looked its items up, all of them (see plan_forward)
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
      Run r;
      do {
        cp_async_wait<kStages - 2>();
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) raw[u] = ring[rd + u * 32];
        rd = rd == (kStages - 1) * kBatch * 32 ? 0 : rd + kBatch * 32;
        issue();
        float2 v[kBatch * P];
        if (n >= kBatch * 32) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) IO::unpack2(raw[u], *reinterpret_cast<float2(*)[P]>(v + u * P));
          add_pairs(r, v, C);
        } else {
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
      float s = r.m == m ? r.s : r.s * ex2_approx((r.m - m) * C);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (lane == 0) a.parts[row * a.most + part] = make_float2(m, s);
    }
    // The batches of nothing at the end: the ring starts the next items where it stands.
    cp_async_wait<0>();
    rd = wr;
    if (a.listed) break;
  }
}

// What the second kernel needs of a row besides its parts.
struct RowInput {
  double w, hit, old_logp, advantage, ref_logp;
};

template <typename T>
__device__ __forceinline__ RowInput row_input(const LossArgs &a, int64_t row) {
  RowInput in = {};
  in.w = a.weight ? (double)__ldcg(a.weight + row) : 1.0 / (double)a.M;
  if (in.w != 0.0) {
    const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
    in.old_logp = (double)__ldcg(a.old_logp + row);
    in.advantage = (double)__ldcg(a.advantage + row);
    if (a.ref_logp) in.ref_logp = (double)__ldcg(a.ref_logp + row);
    // a token outside the vocabulary has no probability: NaN, here and in the loss
    in.hit = tok >= 0 && tok < a.N ? (double)to_f32<T>(__ldcg(static_cast<const T *>(a.z) + row * a.ld + tok))
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
// writes none of them. (Those loads pass by L1, which may be older than that.)
// This kernel is therefore launched directly after loss_rows_kernel, with nothing
// between them, and that one releases its successor nowhere but in pdl_prologue.
template <typename T>
__global__ void __launch_bounds__(kFinishBlock) loss_finish_kernel(LossArgs a) {
  __shared__ double sh[kFinishBlock / 32];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 31;
  const bool wide = a.most > kThreadParts;
  const int64_t per = wide ? kFinishBlock / 32 : kFinishBlock;  // rows of a CTA step
  int64_t row = blockIdx.x * per + (wide ? tid >> 5 : tid);
  RowInput in = {};
  if (row < a.M) in = row_input<T>(a, row);
  pdl_prologue();
  const int parts = (int)a.done[1];
  double sum = 0.0;
  while (row < a.M) {
    Run r;
    if (in.w != 0.0) {
      for (int i = wide ? lane : 0; i < parts; i += wide ? 32 : 1) {
        const float2 p = a.parts[row * a.most + i];
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

constexpr int kGradCtas = 5;  // an SM's

// Measured: 8192 x 131072 bf16 629 us (6.8 TB/s), 4096 x 32003 fp16 with a
// quarter of the rows without weight 79 us (5.8 TB/s); rows at different
// offsets, 4096 x 32003 bf16, 98 us. Bound by memory. Five CTAs an SM, 48
// registers, gain 4% over four on ragged rows (78.9 and 82.1 us). A warp per row
// of 16-bit logits spills 11 registers at that; with four CTAs an SM 16384 x 4096 bf16
// takes 44.5 instead of 45.8 us, but 16384 x 2000 27.4 instead of 26.5 and 16384 x 1000
// fp16 18.5 instead of 17.8.
// G threads (a warp, or the CTA) per part of a row. The vectors are those of
// the output row; SHIFT: the input row lies at another offset past a 16-byte
// boundary, and each of its vectors is cut out of two aligned ones inside the
// row. The elements before and after those vectors are taken one by one.
template <typename T, bool CTA, bool SHIFT>
__global__ void __launch_bounds__(256, kGradCtas) loss_grad_kernel(LossGradArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int U = SHIFT ? 1 : 4;  // vectors under way (SHIFT, 1, 2 and 4: 98, 111 and 106 us for the case above)
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
    // (all of the row's numbers are asked for at once, whichever are used)
    const float coef = a.coef[row];
    const int64_t tok = token_at(a.tokens, a.wide_tokens, row);
    const float2 st = a.stats[row];
    const float A = (float)(gt * (double)coef);
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
    // p = 2^((z - m) C) e^-s: the maximum leaves first, as in the forward. (A power below 2^-126 is 0.)
    const float B = -A * expf(-st.y);
    auto power = [&](float2 z2) {
      const float2 e = mul2(add2(z2, f2(-st.x)), f2(a.C));
      return make_float2(ex2_approx(e.x), ex2_approx(e.y));
    };
    auto one = [&](int64_t j) {
      const float p = power(f2(to_f32<T>(z[j]))).x;
      // two roundings at the token, as in the vectors: the same bits at every offset
      dz[j] = from_f32<T>(j == tok ? __fadd_rn(__fmul_rn(B, p), A) : B * p);
    };
    if (part == 0)
      for (int64_t j = t; j < head; j += G) one(j);
    if (part == a.S - 1)
      for (int64_t j = t; j < rest; j += G) one(a.N - rest + j);
    const uint4 *in = reinterpret_cast<const uint4 *>(z + (head - d));
    auto vec = [&](int64_t i, const uint4 &raw) {
      float2 f[V / 2];
      IO::unpack2(raw, f);
      const int64_t j0 = head + i * V;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) f[e] = mul2(f2(B), power(f[e]));
      if (tok >= j0 && tok < j0 + V) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          f[e].x += j0 + 2 * e == tok ? A : 0.0f;
          f[e].y += j0 + 2 * e + 1 == tok ? A : 0.0f;
        }
      }
      __stcs(out + i, IO::pack2(f));
    };
    int64_t i = b0 + t;
    for (; i + (U - 1) * G < b1; i += U * G) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = a.lines ? __ldcs(in + i + u * G) : in[i + u * G];
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
