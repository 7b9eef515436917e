// Layer norm forward and backward for sm_100a over the rows of an M x N matrix.
//
//   mean = sum_j x_j / N,  var = sum_j (x_j - mean)^2 / N,  rstd = (var + eps)^-1/2
//   y_j  = gamma_j h_j + beta_j,  h_j = (x_j - mean) rstd
//   dx_j = rstd (g_j - c1 - h_j c2),  g_j = gamma_j dy_j,
//          c1 = sum_j g_j / N,  c2 = sum_j g_j h_j / N
//   dgamma_j = sum_i dy_ij h_ij,  dbeta_j = sum_i dy_ij
//
// Both are bound by memory: a row is read once and kept in registers between
// its sums and its outputs. A lane holds E elements of a row (32 in the
// forward over 16-bit rows, else 16: the backward's column sums take twice that
// many registers), the same columns in every row, so gamma and beta are read once and
// the column sums of the backward stay in registers. A row has L lanes: 1 ..
// 32 of a warp (32 / L rows side by side), or a group of whole warps that meet
// at a barrier of their own, several groups to a CTA; rows beyond 512 lanes'
// worth take the kernels for long rows.
#pragma once

#include "dyt_async.cuh"

namespace dyt {
namespace norm {

// How a launch walks the rows: the CTAs' rows side by side, `step` rows further
// at every step. Computed on the host so that the loops keep it out of registers.
struct Walk {
  int64_t M;
  int64_t N;
  int NV;        // vectors of a row (elements, for ragged rows)
  int L;         // lanes of a row
  int rows;      // rows side by side in a CTA
  int step;      // grid x rows
  int64_t inc[4];  // bytes from a row to the one a step later: the inputs, the output
  int64_t fast;  // ragged rows: [fast, M - fast) are copied in whole 16-byte chunks
  int plane;     // bytes of the slots that a warp has for one tensor's rows (read for ragged rows of part of a warp)
  float n, inv_n;
};

struct NormArgs {
  const void *x;
  int64_t ldx;
  const void *gamma;  // NULL: 1
  const void *beta;   // NULL: 0
  void *y;
  int64_t ldy;
  float *mean;  // NULL: not written
  float *rstd;
  int gamma_dt, beta_dt;
  float eps;
  Walk w;
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
  int gamma_dt;
  Walk w;
};

constexpr int kBlock = 512;  // threads of a CTA, at most
// Elements of a row a lane holds.
template <typename T>
__host__ __device__ constexpr int fwd_elems() {
  return sizeof(T) == 4 ? 16 : 32;
}
constexpr int kBwdElems = 16;
// Rows a lane adds in binary32 before its column sums move to binary64: the
// run's rounding is at most 128 * 2^-24 of the sum of its terms' magnitudes.
constexpr int kRunRows = 128;
constexpr int kMaxWarps = 32;

// How many lanes share a row: less than a warp (a power of two), a warp, or a group of warps.
// (kHalf is kPart with 16 lanes, known to the compiler: the offsets of a lane's elements are constants. kCluster: all
// warps of a cluster's CTAs, which have a stretch of the row's columns each; kClusterRows: a group of warps in each of
// them, and several rows side by side.)
enum RowMode { kPart = 0, kWarp = 1, kGroup = 2, kHalf = 3, kCluster = 4, kClusterRows = 5 };
__host__ __device__ constexpr bool shares_warp(int mode) { return mode == kPart || mode == kHalf; }
__host__ __device__ constexpr bool in_cluster(int mode) { return mode == kCluster || mode == kClusterRows; }
__host__ __device__ constexpr bool in_warps(int mode) { return mode == kGroup || in_cluster(mode); }

// Where a thread stands: lane `lane` of the L that share row `mine` of the
// CTA's rows; seg() of those lanes are in this warp, this is number `at` of them.
template <int MODE>
struct Place {
  int L, lane, mine, at;
  __device__ __forceinline__ Place(int L_) : L(MODE == kWarp ? 32 : MODE == kHalf ? 16 : L_) {
    const int t = (int)threadIdx.x;
    if constexpr (MODE == kCluster) {
      mine = 0;
      lane = t;
      at = t & 31;
    } else if constexpr (MODE == kGroup || MODE == kClusterRows) {
      mine = t / L;
      lane = t - mine * L;
      at = t & 31;
    } else {
      lane = at = t & (L - 1);
      mine = MODE == kWarp ? t >> 5 : MODE == kHalf ? t >> 4 : t / L;
    }
  }
  __device__ __forceinline__ int seg() const { return MODE == kPart ? L : MODE == kHalf ? 16 : 32; }
};

// The column of a lane's element i of E. Aligned rows: vectors lane, lane + L,
// ... of 16 bytes; ragged ones: single elements seg apart, within a stretch of
// seg E columns that belongs to the lanes of one warp.
template <int V, int E, bool RAGGED, int MODE>
__device__ __forceinline__ int column(int L, int lane, int i) {
  if constexpr (!RAGGED) return (lane + i / V * L) * V + i % V;
  else if constexpr (in_warps(MODE)) return (lane >> 5) * (32 * E) + (lane & 31) + i * 32;
  else return lane + i * (MODE == kWarp ? 32 : MODE == kHalf ? 16 : L);
}

// ---- parameters ------------------------------------------------------------------
//
// Parameters, partial sums and a row's two means are read by ordinary loads. The read-only path (__ldg, or a
// const __restrict__ pointer) asks that nobody writes the data while the kernel lives, and a programmatic
// launch starts its life before the kernel that writes them has ended; the compiler may also move such a load
// over the wait. (The same times within 1%.)

// Elements col[0 .. V) of a parameter, all loads under way before the first value is used.
template <int V>
__device__ __forceinline__ void params_at(const void *p, int dt, const int64_t (&col)[V], float (&out)[V]) {
  if (dt == DYT_F32) {
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = static_cast<const float *>(p)[col[e]];
    return;
  }
  unsigned short v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = static_cast<const unsigned short *>(p)[col[e]];
#pragma unroll
  for (int e = 0; e < V; ++e)
    out[e] = dt == DYT_BF16 ? __uint_as_float((uint32_t)v[e] << 16) : __half2float(__ushort_as_half(v[e]));
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
  params_at<V>(p, dt, col, out);
}

// gamma or beta for a lane's elements, as pairs (0 past the row's end, where the
// backward relies on it). All loads are under way before the first value is
// used. Aligned rows with parameters on 16-byte boundaries take wide loads.
template <int V, int E, bool RAGGED, int MODE>
__device__ __forceinline__ void load_pairs(const void *p, int dt, const Place<MODE> &at, int N, float none,
                                           float2 (&out)[E / 2]) {
  float f[E];
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = none;
  } else if (!RAGGED && ((uintptr_t)p & 15u) == 0) {
    if (dt == DYT_F32) {
      float4 q[E / 4];
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const int c = column<V, E, RAGGED, MODE>(at.L, at.lane, 4 * i);
        q[i] = static_cast<const float4 *>(p)[(c < N ? c : 0) / 4];
      }
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        f[4 * i] = q[i].x;
        f[4 * i + 1] = q[i].y;
        f[4 * i + 2] = q[i].z;
        f[4 * i + 3] = q[i].w;
      }
    } else {
      uint2 q[E / 4];
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const int c = column<V, E, RAGGED, MODE>(at.L, at.lane, 4 * i);
        q[i] = static_cast<const uint2 *>(p)[(c < N ? c : 0) / 4];
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t w = i & 2 ? q[i / 4].y : q[i / 4].x, u = i & 1 ? w >> 16 : w & 0xFFFFu;
        f[i] = dt == DYT_BF16 ? __uint_as_float(u << 16) : __half2float(__ushort_as_half((unsigned short)u));
      }
    }
  } else {
    int64_t col[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = column<V, E, RAGGED, MODE>(at.L, at.lane, i);
      col[i] = c < N ? c : 0;
    }
    params_at<E>(p, dt, col, f);
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (column<V, E, RAGGED, MODE>(at.L, at.lane, i) >= N) f[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) out[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

// ---- row input and output ------------------------------------------------------------

// A 16-byte asynchronous copy or store under a predicate (a branch around the
// instruction would cost three more).
__device__ __forceinline__ void cp_async16_if(bool p, void *smem_dst, const void *gmem_src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(smem_dst);
  asm volatile("{.reg .pred p; setp.ne.b32 p, %2, 0; @p cp.async.cg.shared.global [%0], [%1], 16;}" ::"r"(d),
               "l"(gmem_src), "r"((int)p)
               : "memory");
}
__device__ __forceinline__ void st16_if(bool p, void *dst, const uint4 &v) {
  asm volatile("{.reg .pred p; setp.ne.b32 p, %5, 0; @p st.global.v4.u32 [%0], {%1,%2,%3,%4};}" ::"l"(dst), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "r"((int)p)
               : "memory");
}

// Ragged rows: slots for the lanes of a row in a warp beyond those that their elements fill: one for the bytes before
// the row's first, the others so that a chunk lies in shared memory as it does in its line of 128 bytes (rows of few
// lanes: in its sector of 32). Where it does not, the copy of every line or sector is split: 100003 x 255 binary32
// backward 58.7 us with one spare slot, 53.6 with sectors kept, 52.6 with lines.
__host__ __device__ constexpr int spare_slots(int L) { return L < 16 ? 2 : 8; }
// 16-byte slots of a block's lanes for one row of one tensor.
template <typename T, int E>
__host__ __device__ constexpr int row_slots(int block, int L, bool ragged) {
  return E * (int)sizeof(T) / 16 * block + (ragged ? block / 32 * (L < 32 ? 32 / L : 1) * spare_slots(L) : 0);
}

// The rows ahead, S - 1 of them under way in a ring of shared memory
// (asynchronous 16-byte copies), read in the order they were copied.
//  - Aligned rows: a thread copies its own vectors and reads them back; no
//    thread reads another's.
//  - RAGGED (rows at any element offset, any N): the lanes of a warp copy the
//    aligned 16-byte chunks that hold their stretch of the row, up to one more than
//    its bytes fill, and read single elements at the row's own offset (neighbouring
//    lanes read neighbouring elements: no bank conflict at any offset, and
//    single-element stores coalesce in the same way). A copied chunk holds at
//    least one byte of the row and up to 15 of those around it; the first and
//    the last `fast` rows, where those may lie outside the tensor, are read from
//    global memory by elements instead.
template <typename T, int E, int TENSORS, int S, bool RAGGED, int MODE>
struct RowFeed {
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int K = E / V;
  unsigned char *mine;      // this thread's slots (RAGGED: its row's in this warp) of stage 0, tensor 0
  const char *at[TENSORS];  // this lane's first vector (RAGGED: its warp's stretch) in the next row to copy
  int need;                 // RAGGED: bytes of the row in this warp's stretch
  int wr = 0, rd = 0;       // byte offsets of the stages to copy to and to read

  // RAGGED: the bits of an address that its place in shared memory keeps.
  static __device__ __forceinline__ uint32_t kept(const Place<MODE> &p) { return spare_slots(p.seg()) * 16 - 1; }
  // Bytes of a warp's slots for one tensor's rows; its ring is S x TENSORS of them.
  static __device__ __forceinline__ int plane(const Walk &w) {
    if constexpr (!RAGGED) return K * 512;
    else if constexpr (MODE == kHalf) return (32 * K + 2 * spare_slots(16)) * 16;
    else if constexpr (MODE != kPart) return (32 * K + spare_slots(32)) * 16;
    else return w.plane;
  }

  __device__ __forceinline__ RowFeed(unsigned char *ring, const T *const (&base)[TENSORS],
                                     const int64_t (&ld)[TENSORS], const Place<MODE> &p, const Walk &w,
                                     int64_t first) {
    const int t = (int)threadIdx.x, N = (int)w.N;
    const int c0 = RAGGED ? column<V, E, true, MODE>(p.L, p.lane - p.at, 0) : p.lane * V;
    mine = ring + (t >> 5) * (S * TENSORS * plane(w)) + (RAGGED ? (t & 31) / p.seg() * (p.seg() * K + spare_slots(p.seg())) : t & 31) * 16;
    need = (N - c0 < p.seg() * E ? N - c0 : p.seg() * E) * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < TENSORS; ++i) at[i] = reinterpret_cast<const char *>(base[i] + first * ld[i] + c0);
    if constexpr (!RAGGED) {  // vectors past the row's end are never copied and stay 0
      for (int i = 0; i < S * TENSORS; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
          *reinterpret_cast<uint4 *>(mine + i * plane(w) + k * 512) = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // Starts the copies of the next row: in: there is one; row: which (RAGGED).
  __device__ __forceinline__ void issue(const Place<MODE> &p, const Walk &w, bool in, int64_t row) {
    if (RAGGED ? row >= w.fast && row < w.M - w.fast : in) {
#pragma unroll
      for (int t = 0; t < TENSORS; ++t) {
        unsigned char *s = mine + wr + t * plane(w);
        if constexpr (!RAGGED) {
#pragma unroll
          for (int k = 0; k < K; ++k)
            cp_async16_if(p.lane + k * p.L < w.NV, s + k * 512, at[t] + (int64_t)(k * p.L) * 16);
        } else {
          const int d = (int)((uintptr_t)at[t] & 15u);
          const char *q = at[t] - d;
          s += (uint32_t)(uintptr_t)q & kept(p);
          const int end = need + d;  // chunks that start before this hold bytes of the row
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int o = (p.at + k * p.seg()) * 16;
            cp_async16_if(o < end, s + o, q + o);
          }
          const int o = p.seg() * K * 16;
          cp_async16_if(p.at == 0 && o < end, s + o, q + o);
        }
      }
    } else if (!RAGGED && shares_warp(MODE)) {  // lanes without a row take part in the warp's sums: with zeros
#pragma unroll
      for (int i = 0; i < TENSORS * K; ++i)
        *reinterpret_cast<uint4 *>(mine + wr + i / K * plane(w) + i % K * 512) = make_uint4(0u, 0u, 0u, 0u);
    }
    cp_async_commit();
    wr = wr == (S - 1) * TENSORS * plane(w) ? 0 : wr + TENSORS * plane(w);
#pragma unroll
    for (int t = 0; t < TENSORS; ++t) at[t] += w.inc[t];
  }

  // The next row to copy is this one (for rows that do not follow at equal steps: with w.inc 0).
  __device__ __forceinline__ void seek(const T *const (&base)[TENSORS], const int64_t (&ld)[TENSORS],
                                       const Place<MODE> &p, int64_t row) {
    const int c0 = RAGGED ? column<V, E, true, MODE>(p.L, p.lane - p.at, 0) : p.lane * V;
#pragma unroll
    for (int i = 0; i < TENSORS; ++i) at[i] = reinterpret_cast<const char *>(base[i] + row * ld[i] + c0);
  }

  // RAGGED: elements g .. g + 7 of every lane of the warp lie inside the row.
  __device__ __forceinline__ bool whole(const Place<MODE> &p, int g) const {
    return (g + 8) * p.seg() * (int)sizeof(T) <= need;
  }

  // RAGGED: none of them does. (Rows of one warp or less with 16 elements a lane fill more than half of them: never.
  // Looked for, empty ones take 100003 x 700 bf16 104 -> 97 us, backward 121 -> 113.)
  __device__ __forceinline__ bool empty(const Place<MODE> &p, int g) const {
    if constexpr (E <= 16 && !in_warps(MODE)) return false;
    else return g * p.seg() * (int)sizeof(T) >= need;
  }

  // The oldest row has landed.
  __device__ __forceinline__ void wait() const {
    cp_async_wait<S - 2>();
    if constexpr (RAGGED) __syncwarp();
  }

  // A lane's elements of row r (the oldest one) of tensor t; 0 past its end.
  __device__ __forceinline__ void read(int t, const T *base, int64_t ld, int64_t r, const Place<MODE> &p, const Walk &w,
                                       float2 (&f)[E / 2]) const {
    const int N = (int)w.N;
    const unsigned char *s = mine + rd + t * plane(w);
    if constexpr (!RAGGED) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        VecIO<T, V>::unpack2(*reinterpret_cast<const uint4 *>(s + k * 512),
                             *reinterpret_cast<float2(*)[V / 2]>(f + k * (V / 2)));
    } else {
      const int c0 = column<V, E, true, MODE>(p.L, p.lane, 0), left = N - c0;  // element i is inside while i seg < left
      T v[E];
      if (r >= w.fast && r < w.M - w.fast) {
        const int d = (int)((uint32_t)(uintptr_t)base + ((uint32_t)r * (uint32_t)ld + (uint32_t)(c0 - p.at)) *
                                                            (uint32_t)sizeof(T)) & kept(p);
        const T *e = reinterpret_cast<const T *>(s + d) + p.at;
#pragma unroll
        for (int g = 0; g < E; g += 8) {
          if (whole(p, g)) {
#pragma unroll
            for (int i = g; i < g + 8; ++i) v[i] = e[i * p.seg()];
          } else if (empty(p, g)) {
#pragma unroll
            for (int i = g; i < g + 8; ++i) v[i] = from_f32<T>(0.0f);
          } else {
#pragma unroll
            for (int i = g; i < g + 8; ++i) v[i] = i * p.seg() < left ? e[i * p.seg()] : from_f32<T>(0.0f);
          }
        }
      } else {
        const T *g = base + (r < w.M ? r * ld + c0 : 0);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = r < w.M && i * p.seg() < left ? g[i * p.seg()] : from_f32<T>(0.0f);
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) f[i] = make_float2(to_f32<T>(v[2 * i]), to_f32<T>(v[2 * i + 1]));
    }
  }
  __device__ __forceinline__ void advance(const Walk &w) {
    rd = rd == (S - 1) * TENSORS * plane(w) ? 0 : rd + TENSORS * plane(w);
  }
};

// A lane's outputs, rounded once to T, to the row that starts at `out`.
template <typename T, int E, bool RAGGED, int MODE, typename Feed>
__device__ __forceinline__ void store_pairs(T *out, const float2 (&f)[E / 2], const Place<MODE> &p, const Feed &feed,
                                            int NV, int N) {
  constexpr int V = 16 / (int)sizeof(T);
  if constexpr (!RAGGED) {
#pragma unroll
    for (int k = 0; k < E / V; ++k)
      st16_if(p.lane + k * p.L < NV, out + (p.lane + k * p.L) * V,
              VecIO<T, V>::pack2(*reinterpret_cast<const float2(*)[V / 2]>(f + k * (V / 2))));
  } else {
    const int c0 = column<V, E, true, MODE>(p.L, p.lane, 0), left = N - c0;
    T *o = out + c0;
#pragma unroll
    for (int g = 0; g < E; g += 8) {
      if (feed.whole(p, g)) {
#pragma unroll
        for (int i = g; i < g + 8; ++i) o[i * p.seg()] = from_f32<T>(i & 1 ? f[i / 2].y : f[i / 2].x);
      } else if (!feed.empty(p, g)) {
#pragma unroll
        for (int i = g; i < g + 8; ++i)
          if (i * p.seg() < left) o[i * p.seg()] = from_f32<T>(i & 1 ? f[i / 2].y : f[i / 2].x);
      }
    }
  }
}

// Rows first, first + step, ... below M.
__device__ __forceinline__ int row_count(int64_t M, int64_t first, int step) {
  return first < M ? (int)((M - first + step - 1) / step) : 0;
}

// ---- sums over a row's lanes -------------------------------------------------------

__device__ __forceinline__ void group_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Over `width` lanes of a warp: every lane gets the same bits.
__device__ __forceinline__ float lanes_sum(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums over a CTA (the kernels for long rows): one barrier; `red` may still be
// read from the call before the last one.
template <int C>
__device__ __forceinline__ void cta_sum(float (&v)[C], float *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = warp_sum(v[c]);
  if (lane == 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) red[c * kMaxWarps + warp] = v[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = warp_sum(lane < warps ? red[c * kMaxWarps + lane] : 0.0f);
}

// s / n for n = N: the product with 1 / n, corrected once. A quotient that binary32 holds comes out exactly (a
// row of equal values whose sum does not round); the sum's rounding stays.
__device__ __forceinline__ float div_n(float s, float n, float inv_n) {
  const float q = s * inv_n;
  return fabsf(q) < __int_as_float(0x7F800000) ? fmaf(fmaf(-q, n, s), inv_n, q) : q;
}

// ---- forward: a row in registers ---------------------------------------------

// Rows in the ring. More gain nothing (3, 4, 5: 16384 x 4096 bf16 48.2, 47.5,
// 47.8 us; 32768 x 8192 171, 187, 187) and leave the SM less L1.
template <typename T>
__host__ __device__ constexpr int fwd_stages() {
  return 3;
}
// 32 elements a lane with gamma and beta in registers spill: beta stays in shared memory then.
template <typename T>
__host__ __device__ constexpr bool fwd_beta_shared() {
  return fwd_elems<T>() == 32;
}
template <typename T>
__host__ __device__ constexpr int fwd_plane(int block, int L, bool ragged) {
  return row_slots<T, fwd_elems<T>()>(block, L, ragged);
}
template <typename T>
__host__ __device__ constexpr size_t fwd_ring(int block, int L, bool ragged) {
  return (size_t)fwd_stages<T>() * fwd_plane<T>(block, L, ragged) * 16;
}
template <typename T>
__host__ __device__ constexpr size_t fwd_smem(int block, int L, bool ragged) {
  return fwd_ring<T>(block, L, ragged) +
         (fwd_beta_shared<T>() ? (size_t)block * fwd_elems<T>() * sizeof(float) : 0);
}

// GROUP: a row takes several warps. A warp sums its part of the row, then the
// squares about that part's own mean, so that one exchange joins the parts:
// M2 = sum_w (M2_w + n_w (mean_w - mean)^2), with no cancellation.
// Measured: 32768 x 8192 bf16 170 us (6.3 TB/s), 16384 x 4096 47 us (5.7 TB/s;
// two barriers a row, 16 elements a lane and one row ahead in registers: 62
// us), 16384 x 2048 fp32 48 us, 100003 x 255 fp32 39 us (5.2 TB/s; 16-byte
// vectors cut out of two chunks with funnel shifts: 73 us). Bound by memory for
// wide rows, by the instructions around a row's sums for narrow ones.
template <typename T, int MODE, bool RAGGED>
__global__ void __launch_bounds__(kBlock, 1) norm_fwd_kernel(NormArgs a) {
  constexpr bool GROUP = MODE == kGroup;
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int E = fwd_elems<T>(), P = E / 2;
  constexpr int S = fwd_stages<T>();
  __shared__ float4 red[2][kBlock / 32];
  extern __shared__ __align__(128) unsigned char dyn[];
  pdl_prologue();
  const Place<MODE> p(a.w.L);
  if (dynamic_smem_bytes() < fwd_smem<T>((int)blockDim.x, p.L, RAGGED)) return;
  const int N = (int)a.w.N;
  const T *const x[1] = {static_cast<const T *>(a.x)};
  const int64_t ld[1] = {a.ldx};
  const int64_t r0 = (int64_t)blockIdx.x * a.w.rows;
  int64_t row = r0 + p.mine;
  const int steps = row_count(a.w.M, r0, a.w.step), left = row_count(a.w.M, row, a.w.step);  // the CTA's, this row's
  RowFeed<T, E, 1, S, RAGGED, MODE> feed(dyn, x, ld, p, a.w, row);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) feed.issue(p, a.w, i < left, row + (int64_t)i * a.w.step);
  constexpr bool BS = fwd_beta_shared<T>();
  // this thread's own slots, 32 apart
  float4 *bslot = reinterpret_cast<float4 *>(dyn + fwd_ring<T>((int)blockDim.x, p.L, RAGGED)) +
                  (threadIdx.x >> 5) * (P / 2 * 32) + (threadIdx.x & 31);
  float2 gam[P], bet[BS ? 1 : P];
  if constexpr (BS) {
    load_pairs<V, E, RAGGED, MODE>(a.beta, a.beta_dt, p, N, 0.0f, gam);
#pragma unroll
    for (int i = 0; i < P / 2; ++i)
      bslot[i * 32] = make_float4(gam[2 * i].x, gam[2 * i].y, gam[2 * i + 1].x, gam[2 * i + 1].y);
  } else {
    load_pairs<V, E, RAGGED, MODE>(a.beta, a.beta_dt, p, N, 0.0f, bet);
  }
  load_pairs<V, E, RAGGED, MODE>(a.gamma, a.gamma_dt, p, N, 1.0f, gam);
  // elements of the row in a warp: in this one, and (GROUP) in warp `wl` of the group
  const float n = a.w.n, inv_n = a.w.inv_n;
  const int warps = GROUP ? p.L / 32 : 1, wl = (int)threadIdx.x & 31, w0 = GROUP ? p.mine * warps : 0;
  auto part = [&](int w) {
    int c = 0;
    if constexpr (RAGGED) {
      c = min(max(N - w * 32 * E, 0), 32 * E);
    } else {
#pragma unroll
      for (int k = 0; k < E / V; ++k) c += min(max(N - (w * 32 + k * p.L) * V, 0), 32 * V);
    }
    return (float)c;
  };
  const float nw = GROUP ? part(p.lane / 32) : n, inv_nw = 1.0f / nw;
  const float nl = GROUP && wl < warps ? part(wl) : 0.0f;
  const bool full = N == p.L * E;  // no lane holds anything past the row's end
  char *out = reinterpret_cast<char *>(static_cast<T *>(a.y) + row * a.ldy);
#pragma unroll 1
  for (int it = 0; it < steps; ++it) {
    const int par = it & 1;
    feed.wait();
    float2 v[P];
    feed.read(0, x[0], ld[0], row, p, a.w, v);
    feed.advance(a.w);
    feed.issue(p, a.w, it + S - 1 < left, row + (int64_t)(S - 1) * a.w.step);
    float2 t0 = v[0], t1 = v[1];  // what lies past the row's end is zero
#pragma unroll
    for (int i = 2; i < P; i += 2) {
      t0 = add2(t0, v[i]);
      t1 = add2(t1, v[i + 1]);
    }
    t0 = add2(t0, t1);
    float s = t0.x + t0.y;
    s = GROUP ? warp_sum(s) : lanes_sum(s, p.L);
    float mean = div_n(s, nw, inv_nw);
    t0 = t1 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int g = 0; g < E; g += 8) {
      if (RAGGED ? feed.whole(p, g) : full) {
#pragma unroll
        for (int i = g / 2; i < g / 2 + 4; ++i) {
          const float2 c = add2(v[i], f2(-mean));
          if (i & 1) t1 = fma2(c, c, t1);
          else t0 = fma2(c, c, t0);
        }
      } else {
#pragma unroll
        for (int i = g / 2; i < g / 2 + 4; ++i) {
          float2 c = add2(v[i], f2(-mean));
          if constexpr (RAGGED) {
            if (column<V, E, RAGGED, MODE>(p.L, p.lane, 2 * i) >= N) c.x = 0.0f;
            if (column<V, E, RAGGED, MODE>(p.L, p.lane, 2 * i + 1) >= N) c.y = 0.0f;
          } else {
            if (p.lane + 2 * i / V * p.L >= a.w.NV) c = make_float2(0.0f, 0.0f);
          }
          if (i & 1) t1 = fma2(c, c, t1);
          else t0 = fma2(c, c, t0);
        }
      }
    }
    t0 = add2(t0, t1);
    float q = t0.x + t0.y;
    q = GROUP ? warp_sum(q) : lanes_sum(q, p.L);
    if constexpr (GROUP) {
      if (wl == 0) red[par][w0 + p.lane / 32] = make_float4(s, q, mean, 0.0f);
      group_barrier(p.mine, p.L);
      // up to 16 warps, one a lane: the lower half of this warp has them
      const float4 o = wl < warps ? red[par][w0 + wl] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      mean = div_n(__shfl_sync(0xFFFFFFFFu, lanes_sum(o.x, 16), 0), n, inv_n);
      const float e = o.z - mean;
      q = __shfl_sync(0xFFFFFFFFu, lanes_sum(wl < warps ? fmaf(e * e, nl, o.y) : 0.0f, 16), 0);
    }
    const float rstd = rsqrtf(fmaf(q, inv_n, a.eps));
    if (it < left) {
      if (p.lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float2 b;
        if constexpr (BS) {
          const float2 *q = reinterpret_cast<const float2 *>(bslot + i / 2 * 32);
          b = q[i & 1];
        } else {
          b = bet[i];
        }
        v[i] = fma2(mul2(add2(v[i], f2(-mean)), f2(rstd)), gam[i], b);
      }
      store_pairs<T, E, RAGGED>(reinterpret_cast<T *>(out), v, p, feed, a.w.NV, N);
    }
    row += a.w.step;
    out += a.w.inc[1];
  }
  cp_async_wait<0>();
}

// ---- forward: rows too long for registers --------------------------------------

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

// One CTA reads each row three times (the second and third time mostly from
// L2): its sum, its centred squares, its outputs. Measured: 4096 x 20480 bf16 255
// us, 4096 x 16384 fp32 196 us (1.3 and 2.7 TB/s of the bytes read and written once).
// One CTA an SM, and each pass waits for the sum of the one before.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(NormArgs a) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][kMaxWarps];
  pdl_prologue();
  const float inv_n = 1.0f / (float)a.w.N;
  const int B = blockDim.x;
  for (int64_t row = blockIdx.x; row < a.w.M; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    T *y = static_cast<T *>(a.y) + row * a.ldy;
    float s[1] = {0.0f};
#pragma unroll 4
    for (int64_t cv = threadIdx.x; cv < a.w.NV; cv += B) {
      float v[V];
      IO::unpack(load_row<T, V>(x + cv * V), v);
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] += v[e];
    }
    cta_sum(s, red[0]);
    const float mean = s[0] / (float)a.w.N;  // a division: a row of equal values whose sum does not round is exact
    float q[1] = {0.0f};
#pragma unroll 4
    for (int64_t cv = threadIdx.x; cv < a.w.NV; cv += B) {
      float v[V];
      IO::unpack(load_row<T, V>(x + cv * V), v);
#pragma unroll
      for (int e = 0; e < V; ++e) q[0] = fmaf(v[e] - mean, v[e] - mean, q[0]);
    }
    cta_sum(q, red[1]);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv_n, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t cv = threadIdx.x; cv < a.w.NV; cv += B) {
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

// Rows in the ring: 3 (32768 x 8192 bf16: 2, 3, 4 take 309, 300, 301 us), 2
// over binary32, whose rows are twice as long (16384 x 2048: 70.4 and 71.9).
template <typename T>
__host__ __device__ constexpr int bwd_stages() {
  return sizeof(T) == 4 ? 2 : 3;
}
// Dynamic shared memory: the ring, then room for the column sums of a run, V
// elements of every lane. (The sums of all elements at the end take the ring's place.)
template <typename T>
__host__ __device__ constexpr size_t bwd_ring(int block, int L, bool ragged) {
  return (size_t)bwd_stages<T>() * 2 * row_slots<T, kBwdElems>(block, L, ragged) * 16;
}
// An element's sums of all lanes lie L + kSumPad apart, so that neighbouring columns lie in different banks.
constexpr int kSumPad = 4;
// Bytes for `per` elements of every lane: a copy per group, or per warp of smaller rows.
__host__ __device__ constexpr size_t sums_smem(int block, int L, int per) {
  return (size_t)(block / (L < 32 ? 32 : L)) * 2 * per * (L + kSumPad) * sizeof(float);
}
template <typename T>
__host__ __device__ constexpr size_t bwd_smem(int block, int L, bool ragged) {
  return bwd_ring<T>(block, L, ragged) + sums_smem(block, L, 16 / (int)sizeof(T));
}
// A thread's share of the ring is at least 192 bytes, and of the sums 128 (1 + kSumPad / L) for
// L >= 32, less for smaller rows: 144 at most.
static_assert(bwd_ring<__half>(32, 32, false) >= sums_smem(32, 32, kBwdElems) &&
                  bwd_ring<float>(32, 32, false) >= sums_smem(32, 32, kBwdElems),
              "the last column sums take the ring's place");

// The column sums of one run of rows, added over the CTA's rows in a fixed
// order and moved to its partial sums in binary64 (added to them after the
// first run). Rows side by side in a warp are added by a butterfly first; `sh`
// then holds a copy per warp (rows within a warp) or per group, PER elements of
// every lane at a time.
template <int V, int E, int PER, bool RAGGED, int MODE>
__device__ __forceinline__ void flush_columns(const NormGradArgs &a, float2 (&dg)[E / 2], float2 (&db)[E / 2],
                                              const Place<MODE> &p, bool first, float *sh) {
  double *pg = a.parts + (int64_t)blockIdx.x * 2 * a.w.N;
  const int N = (int)a.w.N;
  const int copies = MODE != kGroup ? (int)blockDim.x / 32 : a.w.rows;
  const int copy = MODE != kGroup ? (int)threadIdx.x >> 5 : p.mine;
  const int stride = p.L + kSumPad, plane = 2 * PER * stride;
  // element e of lane `lane`, column c: which = 0 dgamma, 1 dbeta
  auto add = [&](int which, int e, int lane, int c) {
    if (c >= N) return;
    const float *q = sh + (which * PER + e) * stride + lane;
    double t[2] = {0.0, 0.0};
    for (int w = 0; w + 1 < copies; w += 2) {
      t[0] += (double)q[w * plane];
      t[1] += (double)q[(w + 1) * plane];
    }
    if (copies & 1) t[0] += (double)q[(copies - 1) * plane];
    double *o = pg + (int64_t)which * a.w.N + c;
    *o = first ? t[0] + t[1] : *o + (t[0] + t[1]);
  };
#pragma unroll
  for (int k = 0; k < E; k += PER) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int i = (k + e) / 2;
      float u = e & 1 ? dg[i].y : dg[i].x, w = e & 1 ? db[i].y : db[i].x;
      for (int o = p.seg(); o < 32; o <<= 1) {
        u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
        w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
      }
      if (MODE != kPart || ((int)threadIdx.x & 31) < p.L) {
        sh[copy * plane + e * stride + p.lane] = u;
        sh[copy * plane + (PER + e) * stride + p.lane] = w;
      }
    }
    __syncthreads();
    // neighbouring threads take neighbouring columns
    if constexpr (RAGGED) {
      for (int q = p.mine; q < 2 * PER; q += a.w.rows) {
        const int which = q >= PER, e = q - which * PER;
        add(which, e, p.lane, column<V, E, true, MODE>(p.L, p.lane, k + e));
      }
    } else {
#pragma unroll
      for (int v = 0; v < PER; v += V) {
        for (int j = threadIdx.x; j < 2 * V * p.L; j += blockDim.x) {
          const int which = j >= V * p.L, r = j - which * V * p.L;
          add(which, v + r % V, r / V, (k + v) * p.L + r);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dg[i] = db[i] = make_float2(0.0f, 0.0f);
}

// Two sums over a warp at once: the halves of the warp take one each (the upper
// half the second), in every lane of the half.
__device__ __forceinline__ float half_sums(float u, float w) {
  const bool up = (threadIdx.x & 16) != 0;
  float v = (up ? w : u) + __shfl_xor_sync(0xFFFFFFFFu, up ? u : w, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ void swap_halves(float v, float &u, float &w) {
  const bool up = (threadIdx.x & 16) != 0;
  const float other = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
  u = up ? other : v;
  w = up ? v : other;
}

// A row's two sums meet at one barrier (a group) or in a butterfly that gives
// each half of the warp one of them. Measured: 32768 x 8192 bf16 296 us with the
// sum of the partials (5.4 TB/s), 16384 x 4096 77 us, 16384 x 2048 fp32 68 us,
// 100003 x 255 fp32 63 us, 8191 x 1001 fp16 20.5 us (about 4 of them the launch
// and the column sums, 4 the second kernel). Bound by the arithmetic's latency: 16 warps hold all
// registers, and issue half of the time (300 instructions a warp and row). Not
// kept: two rows at a barrier (290 us at full clock, 307 instead of 305 under
// the power cap), 32 elements a lane in 8 warps (329 us), 8 in 32 (more
// instructions than they hide).
template <typename T, int MODE, bool RAGGED>
__global__ void __launch_bounds__(kBlock, 1) norm_bwd_kernel(NormGradArgs a) {
  constexpr bool GROUP = MODE == kGroup;
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int E = kBwdElems, P = E / 2;
  constexpr int S = bwd_stages<T>();
  __shared__ float red[2][2 * kBlock / 32];
  extern __shared__ __align__(128) unsigned char dyn[];
  pdl_prologue();
  const Place<MODE> p(a.w.L);
  if (dynamic_smem_bytes() < bwd_smem<T>((int)blockDim.x, p.L, RAGGED)) return;
  float *sh = reinterpret_cast<float *>(dyn + bwd_ring<T>((int)blockDim.x, p.L, RAGGED));
  const int N = (int)a.w.N;
  const T *const src[2] = {static_cast<const T *>(a.x), static_cast<const T *>(a.dy)};
  const int64_t ld[2] = {a.ldx, a.lddy};
  const int64_t r0 = (int64_t)blockIdx.x * a.w.rows;
  int64_t row = r0 + p.mine;
  const int steps = row_count(a.w.M, r0, a.w.step), left = row_count(a.w.M, row, a.w.step);  // the CTA's, this row's
  RowFeed<T, E, 2, S, RAGGED, MODE> feed(dyn, src, ld, p, a.w, row);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) feed.issue(p, a.w, i < left, row + (int64_t)i * a.w.step);
  // The next row's statistics, loaded one row ahead and used as they are: past
  // its last row a lane stays at that row (at M - 1 if it has none), so that
  // nothing waits for the loads before the next row.
  int64_t stat = left > 0 ? row : a.w.M - 1;
  float nmean = a.mean[stat], nrstd = a.rstd[stat];
  float2 gam[P], dg[P], db[P];
  load_pairs<V, E, RAGGED, MODE>(a.gamma, a.gamma_dt, p, N, 1.0f, gam);
#pragma unroll
  for (int i = 0; i < P; ++i) dg[i] = db[i] = make_float2(0.0f, 0.0f);
  const float inv_n = a.w.inv_n;
  const int warps = GROUP ? p.L / 32 : 1, wl = (int)threadIdx.x & 31, w0 = GROUP ? p.mine * warps : 0;
  char *out = reinterpret_cast<char *>(static_cast<T *>(a.dx) + row * a.lddx);
  const bool full = N == p.L * E;  // no lane holds anything past the row's end
  bool first = true;
  int run = 0;
#pragma unroll 1
  for (int it = 0; it < steps; ++it) {
    const bool in = it < left;
    const float mean = in ? nmean : 0.0f, rstd = in ? nrstd : 0.0f;
    if (MODE != kPart && !in) break;  // whole warps without a row: only at the CTA's last step
    feed.wait();
    float2 h[P], d[P];
    feed.read(0, src[0], ld[0], row, p, a.w, h);
    feed.read(1, src[1], ld[1], row, p, a.w, d);
    feed.advance(a.w);
    feed.issue(p, a.w, it + S - 1 < left, row + (int64_t)(S - 1) * a.w.step);
    if (it + 1 < left) stat += a.w.step;
    nmean = a.mean[stat];
    nrstd = a.rstd[stat];
    // Past the row's end d and gamma are 0, so that nothing there enters a sum that is used, as long as what
    // they are multiplied with is finite. h = -mean rstd may not be (a row far from 0 with a small variance).
    // Ragged rows therefore sum the products of gamma dy rstd and x - mean, which costs nothing there; aligned
    // ones sum once more without the lanes' parts past the end if it is infinite. (16384 x 512 fp16 15.7 us, the
    // ragged rows' way 16.3; 8191 x 1001 fp16 20.5 us, the aligned rows' way 22.3.)
    float2 s1[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)}, s2[2] = {s1[0], s1[0]};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 c = add2(h[i], f2(-mean));
      h[i] = mul2(c, f2(rstd));
      dg[i] = fma2(d[i], h[i], dg[i]);
      db[i] = add2(db[i], d[i]);
      d[i] = mul2(gam[i], d[i]);
      if constexpr (RAGGED) d[i] = mul2(d[i], f2(rstd));
      s1[i & 1] = add2(s1[i & 1], d[i]);
      s2[i & 1] = fma2(d[i], RAGGED ? c : h[i], s2[i & 1]);
    }
    if (!RAGGED && !full && fabsf(mean * rstd) == __int_as_float(0x7F800000)) {
      s2[0] = s2[1] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (p.lane + 2 * i / V * p.L < a.w.NV) s2[i & 1] = fma2(d[i], h[i], s2[i & 1]);
    }
    s1[0] = add2(s1[0], s1[1]);
    s2[0] = add2(s2[0], s2[1]);
    float c1 = s1[0].x + s1[0].y, c2 = s2[0].x + s2[0].y;
    if constexpr (GROUP) {
      const int par = it & 1;
      float v = half_sums(c1, c2);
      if ((wl & 15) == 0) red[par][2 * (w0 + p.lane / 32) + (wl >> 4)] = v;
      group_barrier(p.mine, p.L);
      v = (wl & 15) < warps ? red[par][2 * (w0 + (wl & 15)) + (wl >> 4)] : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      swap_halves(v, c1, c2);
    } else if constexpr (MODE == kWarp) {
      swap_halves(half_sums(c1, c2), c1, c2);
    } else {
      c1 = lanes_sum(c1, p.L);
      c2 = lanes_sum(c2, p.L);
    }
    if (MODE != kPart || in) {
      c1 *= inv_n;
      c2 *= inv_n;
      if constexpr (RAGGED) {  // c1 has the factor rstd already, and c2 lacks it here
        c2 *= rstd;
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = fma2(h[i], f2(-c2), add2(d[i], f2(-c1)));
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = mul2(f2(rstd), add2(d[i], fma2(h[i], f2(-c2), f2(-c1))));
      }
      store_pairs<T, E, RAGGED>(reinterpret_cast<T *>(out), d, p, feed, a.w.NV, N);
    }
    row += a.w.step;
    out += a.w.inc[2];
    if (++run == kRunRows && it + 1 < steps) {
      flush_columns<V, E, V, RAGGED>(a, dg, db, p, first, sh);
      first = false;
      run = 0;
    }
  }
  // The last run, all elements at once where the ring was: every warp of the
  // CTA is here, also one that left at the last step.
  cp_async_wait<0>();
  __syncthreads();
  flush_columns<V, E, E, RAGGED>(a, dg, db, p, first, reinterpret_cast<float *>(dyn));
}

// ---- backward: rows too long for registers ------------------------------------------

// c1 and c2 of each row, one CTA per row. (The rows are then read once more:
// 5 passes over the data instead of 3.) Measured, with the column pass and the sum
// of the partials: 8192 x 12288 bf16 311 us, 4096 x 16384 bf16 208, fp32 247 (1.9 to 3.3
// TB/s of the bytes read and written once).
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_bwd_rows_kernel(NormGradArgs a, float2 *c12) {
  using IO = VecIO<T, V>;
  __shared__ float red[2][2 * kMaxWarps];
  pdl_prologue();
  const float inv_n = 1.0f / (float)a.w.N;
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.w.M; row += gridDim.x, par ^= 1) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int64_t cv = threadIdx.x; cv < a.w.NV; cv += blockDim.x) {
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
    cta_sum(c, red[par]);
    if (threadIdx.x == 0) c12[row] = make_float2(c[0] * inv_n, c[1] * inv_n);
  }
}

// dx and the column sums: a CTA takes blockDim.x vector-columns (blockIdx.x)
// of every gridDim.y-th row.
template <typename T, int V>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(NormGradArgs a, const float2 *c12) {
  using IO = VecIO<T, V>;
  pdl_prologue();
  const int64_t cv = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (cv >= a.w.NV) return;
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
  for (int64_t row = blockIdx.y; row < a.w.M; row += gridDim.y) {
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
  double *pg = a.parts + (int64_t)blockIdx.y * 2 * a.w.N + cv * V, *pb = pg + a.w.N;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    pg[e] = sg[e] + (double)dg[e];
    pb[e] = sb[e] + (double)db[e];
  }
}

// ---- backward: the parameters' gradients ---------------------------------------------

constexpr int kSumCols = 32, kSumLanes = 16, kSumBatch = 10;

// The CTAs' column sums added in binary64 in a fixed order (lane l takes
// partials l, l + 16, ..., ten loads under way at a time) and rounded once. The
// sums go by halves: one binary64 addition after the other cost 1.4 us more. blockIdx.y < SETS: 0 = dgamma, 1 = dbeta.
template <int SETS>
__global__ void __launch_bounds__(kSumCols *kSumLanes)
    norm_finalize_kernel(const double *parts, int nparts, int64_t N, void *dgamma, int gamma_dt,
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
    for (int i = lane; i < nparts; i += kSumLanes * kSumBatch) {
      double v[kSumBatch];
#pragma unroll
      for (int b = 0; b < kSumBatch; ++b) {
        const int j = i + b * kSumLanes;
        v[b] = j < nparts ? p[(int64_t)j * SETS * N] : 0.0;
      }
#pragma unroll
      for (int s = 1; s < kSumBatch; s <<= 1)  // by halves: few additions wait for one another
#pragma unroll
        for (int b = 0; b + s < kSumBatch; b += 2 * s) v[b] += v[b + s];
      t += v[0];
    }
  }
  sh[lane][c] = t;
  __syncthreads();
  if (lane == 0 && col < N) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int l = 0; l < kSumLanes; ++l) s[l & 3] += sh[l][c];
    store_param(out, blockIdx.y ? beta_dt : gamma_dt, col, (s[0] + s[1]) + (s[2] + s[3]));
  }
}

}  // namespace norm
}  // namespace dyt
