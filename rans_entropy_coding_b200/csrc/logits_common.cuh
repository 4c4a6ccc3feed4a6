// logits_common.cuh -- reading rows of logits with their adjustments
// (penalties, biases, masks), shared by the kernels of logits.cu, tokens.cu,
// distill.cu and beam.cu (and, for rows of any numbers, mxfp4.cu).
//
// Rows may start anywhere an element may (odd vocabularies, strided views).
// A kernel walks a row in vectors of 16 bytes at 16-byte aligned addresses:
// element v sits at u = v + shift, where shift is the row's distance in
// elements from the aligned address below it; only the first and the last
// vector of a row are partial, and those are read element by element.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rans_b200.h"

namespace rb {

constexpr float kNegInf = -__builtin_huge_valf();

template <typename T>
struct VecOf {
  static constexpr int N = 16 / (int)sizeof(T);
};

__device__ __forceinline__ float logit_float(float x) { return x; }
__device__ __forceinline__ float logit_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float logit_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T float_logit(float x);
template <>
__device__ __forceinline__ float float_logit<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half float_logit<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 float_logit<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ void unpack16(const uint4 &q, float (&z)[4], float) {
  z[0] = __uint_as_float(q.x);
  z[1] = __uint_as_float(q.y);
  z[2] = __uint_as_float(q.z);
  z[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack16(const uint4 &q, float (&z)[8], __half) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    z[2 * i] = f.x;
    z[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack16(const uint4 &q, float (&z)[8], __nv_bfloat16) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = __uint_as_float(w[i] << 16);
    z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack16(const float (&z)[4], float) {
  return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]),
                    __float_as_uint(z[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&z)[8], __half) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(z[2 * i], z[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack16(const float (&z)[8], __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// max that keeps a NaN, so that one test per row finds it.
__device__ __forceinline__ float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// The larger (NaN if either is) and the smaller of packed pairs.
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b, __half) {
  uint32_t c;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b, __half) {
  uint32_t c;
  asm("min.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t c;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t c;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// The larger of packed pairs; a NaN gives way.
__device__ __forceinline__ uint32_t pair_most(uint32_t a, uint32_t b, __half) {
  uint32_t c;
  asm("max.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
__device__ __forceinline__ uint32_t pair_most(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t c;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// One row as the kernels walk it.
template <typename T>
struct Row {
  const T *at0;  // 16-byte aligned: element u sits at at0 + u
  int shift;     // u of element 0
  int vocab;

  __device__ __forceinline__ Row(const void *data, int64_t r, int64_t stride, int v) {
    const T *p = static_cast<const T *>(data) + r * stride;
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    at0 = p - shift;
    vocab = v;
  }
  __device__ __forceinline__ int end() const { return shift + vocab; }
  __device__ __forceinline__ bool whole(int u0) const {
    return u0 >= shift && u0 + VecOf<T>::N <= end();
  }
  // The vector at u0 (a multiple of its size); elements off the row's ends
  // read `fill`.
  __device__ __forceinline__ void load(int u0, float (&z)[VecOf<T>::N], float fill) const {
    if (whole(u0)) {
      unpack16(*reinterpret_cast<const uint4 *>(at0 + u0), z, T());
    } else {
#pragma unroll
      for (int i = 0; i < VecOf<T>::N; ++i)
        z[i] = u0 + i >= shift && u0 + i < end() ? logit_float(at0[u0 + i]) : fill;
    }
  }
};

// N elements from p on, any alignment of their type; those at or past `end`
// read 0.  Vectors off the 16-byte boundaries are joined from the two aligned
// ones that hold them.
template <typename T>
__device__ __forceinline__ uint4 load_joined(const T *first, const T *p, const T *end) {
  constexpr int N = VecOf<T>::N;
  const int past = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
  const T *a = p - past;
  if (past == 0 && p + N <= end) return *reinterpret_cast<const uint4 *>(p);
  if (past != 0 && a >= first && a + 2 * N <= end) {
    const uint4 lo = reinterpret_cast<const uint4 *>(a)[0];
    const uint4 hi = reinterpret_cast<const uint4 *>(a)[1];
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int bytes = past * (int)sizeof(T), words = bytes >> 2;
    if (words & 1) {
#pragma unroll
      for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
    }
    if (words & 2) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2 < 8 ? i + 2 : 7];
    }
    if (bytes & 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  float z[N];
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = p + i < end ? logit_float(p[i]) : 0.0f;
  return pack16(z, T());
}

// STREAM: the result is not to push anything out of L2.
template <bool STREAM>
__device__ __forceinline__ void store16(void *at, uint4 p) {
  if (STREAM) __stcs(static_cast<uint4 *>(at), p);
  else *static_cast<uint4 *>(at) = p;
}

// Stores a warp's tile: K vector rows of packed elements, p[k] of lane l at
// u + (32 k + l) N, to o[u ...], at any alignment.  Where o's 16-byte boundaries
// fall inside the vectors (odd vocabularies: the rows of a contiguous result
// start anywhere), a lane joins its vector's tail to the head of the next one,
// lane 31 to lane 0's of the next vector row, and stores that; what is left at
// the tile's two ends goes out as N single elements, a lane each.  (Joining each
// vector row by itself cost 15 instructions an element, half of a kernel's.)
// `inside`: the whole tile is to be stored; else elements from <= u < to are.
template <bool STREAM, int K, typename T>
__device__ __forceinline__ void store_tile(T *o, int u, const uint4 (&p)[K], bool inside, int from,
                                           int to) {
  constexpr int N = VecOf<T>::N;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int past = (int)((reinterpret_cast<uintptr_t>(o + u) & 15) / sizeof(T));
  if (past == 0 || !inside) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u0 = u + (32 * k + lane) * N;
      if (past == 0 && (inside || (u0 >= from && u0 + N <= to))) {
        store16<STREAM>(o + u0, p[k]);
      } else {
        const T *e = reinterpret_cast<const T *>(&p[k]);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (u0 + i >= from && u0 + i < to) o[u0 + i] = e[i];
      }
    }
    return;
  }
  const int skip = N - past;  // elements up to the boundary; the same for the row
  {
    // lane 0's first `skip` elements and lane 31's last others
    const uint32_t a[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
    const uint32_t b[4] = {p[K - 1].x, p[K - 1].y, p[K - 1].z, p[K - 1].w};
    const int i = lane * (int)sizeof(T) / 4;  // its word
    uint32_t x = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t f = __shfl_sync(kAll, a[j], 0), l = __shfl_sync(kAll, b[j], 31);
      if (j == i) x = lane < skip ? f : l;
    }
    if (lane < N) {
      T *at = o + u + (lane < skip ? lane : (32 * K - 1) * N + lane);
      if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t *>(at) = x;
      else *reinterpret_cast<uint16_t *>(at) = (uint16_t)(lane & 1 ? x >> 16 : x);
    }
  }
  const int words = skip * (int)sizeof(T) / 4;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint4 n = k + 1 < K && lane == 0 ? p[k + 1 < K ? k + 1 : k] : p[k];
    uint32_t w[8] = {p[k].x, p[k].y, p[k].z, p[k].w, n.x, n.y, n.z, n.w};
#pragma unroll
    for (int i = 4; i < 8; ++i) w[i] = __shfl_sync(kAll, w[i], lane + 1);  // (31: lane 0's)
    if (words & 1) {
#pragma unroll
      for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
    }
    if (words & 2) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
    }
    if (sizeof(T) == 2 && (skip & 1)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    if (k + 1 < K || lane < 31)
      store16<STREAM>(o + u + (32 * k + lane) * N + skip, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// ---------------------------------------------------------- adjustments --
// One row's adjustments, resolved from rans_adjust.  Kernels keep it in shared
// memory: it is the same for all threads, and most of it is read for touched
// tokens alone.
struct RowAdjust {
  float repetition, frequency, presence, inv_temperature;
  const int32_t *history;  // the row's window
  int64_t history_n;
  const int32_t *bias_ids;
  const float *bias_values;
  int64_t bias_n;
  const uint32_t *mask;  // the row's words, or NULL
  int mask_words;

  __device__ __forceinline__ bool touches() const { return history_n > 0 || bias_n > 0; }
};

__device__ __forceinline__ int64_t clip_window(const int64_t *begin, const int64_t *end,
                                               int64_t r, int64_t len, int64_t &b) {
  b = begin[r];
  int64_t e = end[r];
  b = b < 0 ? 0 : (b > len ? len : b);
  e = e > len ? len : e;
  return e > b ? e - b : 0;
}

__device__ __forceinline__ RowAdjust row_adjust(const rans_adjust &a, int64_t r, int vocab) {
  RowAdjust x;
  x.repetition = a.repetition;
  x.frequency = a.frequency;
  x.presence = a.presence;
  x.inv_temperature = a.inv_temperature;
  if (a.params) {
    const float *p = a.params + 4 * r;
    x.repetition = p[0];
    x.frequency = p[1];
    x.presence = p[2];
    x.inv_temperature = p[3];
  }
  int64_t b = 0;
  x.history = nullptr;
  x.history_n = 0;
  if (a.history) {
    x.history_n = clip_window(a.history_begin, a.history_end, r, a.history_len, b);
    x.history = a.history + b;
  }
  x.bias_ids = nullptr;
  x.bias_values = nullptr;
  x.bias_n = 0;
  if (a.bias_ids) {
    x.bias_n = clip_window(a.bias_begin, a.bias_end, r, a.bias_len, b);
    x.bias_ids = a.bias_ids + b;
    x.bias_values = a.bias_values + b;
  }
  x.mask = a.mask ? a.mask + r * a.mask_stride : nullptr;
  x.mask_words = (vocab + 31) >> 5;
  return x;
}

// Which tokens a row's history and biases touch, and their adjusted logits, in
// shared memory.  They are few, but spread out: handled where they are met,
// nearly every warp would stop for one in every vector (49 instructions per
// logit, measured on rows of 50,000 tokens with 300 touched).  So they are
// gathered and adjusted first, the kernels' main walks leave them out, and what
// they add comes from the table, a token per thread.
// The table is a hash that covers up to kHashSpan tokens at once.  If they
// have more than kHashTokens touched ones among them, there is a cell per token
// instead, for kTouchSpan tokens at a time.
constexpr int kHashSlots = 4096;
constexpr int kHashTokens = kHashSlots * 7 / 8;
constexpr int kHashSpan = 1 << 17;
constexpr int kTouchSpan = 8192;

struct __align__(16) TouchTable {
  union {
    struct {
      int32_t key[kHashSlots];    // place in the span, or -1
      uint32_t count[kHashSlots]; // occurrences; then the adjusted logit
      uint32_t bias[kHashSlots];  // 1 + the last entry's position in the row's list
      uint16_t used[kHashTokens]; // the slots in use, in any order
    } hash;
    struct {
      uint32_t bits[kTouchSpan / 32];  // touched tokens
      uint32_t count[kTouchSpan];
      uint32_t bias[kTouchSpan];
    } cells;
  };
  int u_lo, span;  // covers u in [u_lo, u_lo + span)
  int n_used;      // touched tokens in the hash; more than kHashTokens: too many
  int shift;       // 32 - log2(slots)
  bool dense;      // a cell per token

  __device__ __forceinline__ uint32_t slot(int k) const {
    return (uint32_t)k * 2654435761u >> shift;  // Fibonacci hashing
  }
  __device__ __forceinline__ uint32_t next(uint32_t s) const {
    return (s + 1) & ((1u << (32 - shift)) - 1u);
  }
};

// body(u, its adjusted logit) for every touched token of the table, spread over
// the block's threads.
template <class Body>
__device__ __forceinline__ void each_touched(TouchTable &t, int tid, int threads, Body body) {
  if (!t.dense) {
    for (int i = tid; i < t.n_used; i += threads) {
      const int s = t.hash.used[i];
      body(t.u_lo + t.hash.key[s], __uint_as_float(t.hash.count[s]));
    }
  } else {
    for (int w = tid; w < kTouchSpan / 32; w += threads)
      for (uint32_t b = w * 32 < t.span ? t.cells.bits[w] : 0u; b != 0; b &= b - 1) {
        const int k = w * 32 + __ffs(b) - 1;
        body(t.u_lo + k, __uint_as_float(t.cells.count[k]));
      }
  }
}

// The adjusted logit of a token that may be touched; -inf if it is not.
__device__ __forceinline__ float touched_logit(TouchTable &t, int u) {
  const int k = u - t.u_lo;
  if (k < 0 || k >= t.span) return kNegInf;
  if (t.dense)
    return t.cells.bits[k >> 5] >> (k & 31) & 1 ? __uint_as_float(t.cells.count[k]) : kNegInf;
  for (uint32_t s = t.slot(k); t.hash.key[s] != -1; s = t.next(s))  // (never full)
    if (t.hash.key[s] == k) return __uint_as_float(t.hash.count[s]);
  return kNegInf;
}

// Bits of the row's tokens u_lo .. u_lo + span - 1 that the mask leaves; 0 off
// the row's ends.  `mask` may be NULL.  No barrier.
template <typename T>
__device__ __forceinline__ void fill_mask(uint32_t *ok, const uint32_t *mask, int words,
                                          const Row<T> &row, int u_lo, int span, int tid,
                                          int threads) {
  for (int i = tid; i < (span + 31) / 32; i += threads) {
    const int u = u_lo + 32 * i, v = u - row.shift;
    uint32_t b = ~0u;
    if (mask) {
      const int w = v >> 5;
      b = __funnelshift_r(mask[min(max(w, 0), words - 1)], mask[min(max(w + 1, 0), words - 1)],
                          v & 31);
    }
    if (v < 0) b &= ~0u << -v;
    if (u + 32 > row.end()) b &= ~0u >> (u + 32 - row.end());
    ok[i] = b;
  }
}

// Fills the table from u_lo on, up to u_hi, and returns the tokens it covers.
// `dense` is a block's memory of having met too many touched tokens (false at
// first).  `ok`, if given, gets the bits of the tokens covered that the mask
// leaves and nothing touches.  Called by `threads` threads of the block that meet at `barrier`,
// which also begins and ends it.  Counts
// come from integer adds, maxima and ors: what a token finds does not depend on
// the threads' order.
template <typename T, class Barrier>
__device__ __forceinline__ int fill_touch(TouchTable &t, const RowAdjust &a, const Row<T> &row,
                                          int u_lo, int u_hi, bool &dense, uint32_t *ok, int tid,
                                          int threads, Barrier barrier) {
  const int64_t n = a.history_n + a.bias_n;
  int span = min(kHashSpan, u_hi - u_lo);
  // body(place in the span, entry) for the window's entries, kFlight loads in
  // flight per thread
  constexpr int kFlight = 8;
  auto window = [&](auto body) {
    for (int64_t i0 = tid; i0 < n; i0 += kFlight * threads) {
      int v[kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int64_t i = i0 + j * threads;
        v[j] = i >= n ? -1 : i < a.history_n ? a.history[i] : a.bias_ids[i - a.history_n];
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int k = v[j] + row.shift - u_lo;
        if (v[j] >= 0 && v[j] < row.vocab && k >= 0 && k < span) body(k, i0 + j * threads);
      }
    }
  };
  // what the token at place k needs from memory, and its adjusted logit
  struct Raw {
    float z, bias;
    uint32_t mask;
  };
  auto raw_of = [&](int k, uint32_t entry) {
    const int u = u_lo + k, v = u - row.shift;
    return Raw{logit_float(row.at0[u]), entry > 0 ? a.bias_values[entry - 1] : 0.0f,
               a.mask ? a.mask[v >> 5] >> (v & 31) : 1u};
  };
  auto adjusted = [&](const Raw &w, uint32_t count, uint32_t entry) {
    float z = w.z;
    if (count > 0) {
      z = z > 0.0f ? __fdiv_rn(z, a.repetition) : __fmul_rn(z, a.repetition);
      z = __fsub_rn(z, __fadd_rn(__fmul_rn(__uint2float_rn(count), a.frequency), a.presence));
    }
    if (entry > 0) z = __fadd_rn(z, w.bias);
    return __float_as_uint(w.mask & 1 ? z : kNegInf);
  };

  if (!dense) {
    // twice the window's entries, up to kHashSlots
    int log2 = 6;
    while (log2 < 12 && (1 << log2) < 2 * n) ++log2;
    const int slots = 1 << log2;
    barrier();
    if (tid == 0) {
      t.u_lo = u_lo;
      t.span = span;
      t.n_used = 0;
      t.shift = 32 - log2;
      t.dense = false;
    }
    if (ok) fill_mask(ok, a.mask, a.mask_words, row, u_lo, span, tid, threads);
    for (int i = tid; i < slots; i += threads) {
      t.hash.key[i] = -1;
      t.hash.count[i] = 0;
      t.hash.bias[i] = 0;
    }
    barrier();
    window([&](int k, int64_t i) {
      uint32_t s = t.slot(k);
      int old = 0, tries = 0;
      // (a full table ends the search)
      while (tries++ < slots && (old = atomicCAS(&t.hash.key[s], -1, k)) != -1 && old != k)
        s = t.next(s);
      if (old == -1) {
        const int at = atomicAdd(&t.n_used, 1);
        if (at < kHashTokens) t.hash.used[at] = (uint16_t)s;
        if (ok) atomicAnd(&ok[k >> 5], ~(1u << (k & 31)));
      }
      if (old != -1 && old != k) return;
      if (i < a.history_n) atomicAdd(&t.hash.count[s], 1u);
      else atomicMax(&t.hash.bias[s], (uint32_t)(i - a.history_n) + 1u);
    });
    barrier();
    dense = t.n_used > kHashTokens;
    if (!dense) {
      // (four tokens' logits in flight per thread)
      for (int i0 = tid; i0 < t.n_used; i0 += 4 * threads) {
        Raw raw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * threads < t.n_used) {
            const int s = t.hash.used[i0 + j * threads];
            raw[j] = raw_of(t.hash.key[s], t.hash.bias[s]);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * threads < t.n_used) {
            const int s = t.hash.used[i0 + j * threads];
            t.hash.count[s] = adjusted(raw[j], t.hash.count[s], t.hash.bias[s]);
          }
      }
      barrier();
      return span;
    }
  }
  span = min(kTouchSpan, u_hi - u_lo);
  uint32_t *bits = t.cells.bits;
  barrier();
  if (tid == 0) {
    t.u_lo = u_lo;
    t.span = span;
    t.dense = true;
  }
  for (int i = tid; i < (span + 31) / 32; i += threads) bits[i] = 0;
  for (int i = tid; i < span; i += threads) {
    t.cells.count[i] = 0;
    t.cells.bias[i] = 0;
  }
  if (ok) fill_mask(ok, a.mask, a.mask_words, row, u_lo, span, tid, threads);
  barrier();
  window([&](int k, int64_t i) {
    if (i < a.history_n) atomicAdd(&t.cells.count[k], 1u);
    else atomicMax(&t.cells.bias[k], (uint32_t)(i - a.history_n) + 1u);
    atomicOr(&bits[k >> 5], 1u << (k & 31));
  });
  barrier();
  for (int w = tid; w < (span + 31) / 32; w += threads) {
    if (ok) ok[w] &= ~bits[w];
    for (uint32_t b = bits[w]; b != 0; b &= b - 1) {
      const int k = w * 32 + __ffs(b) - 1;
      t.cells.count[k] =
          adjusted(raw_of(k, t.cells.bias[k]), t.cells.count[k], t.cells.bias[k]);
    }
  }
  barrier();
  return span;
}

// Mask bits of a warp's vectors, lane l's N tokens from v0 + l * N on: a few
// lanes load the words, each word once, and the others get theirs by shuffles.
// (v0 may be below 0 by part of a vector, whose bits mean nothing there.)
template <int N>
__device__ __forceinline__ uint32_t load_mask(const uint32_t *mask, int words, int v0, int lane) {
  const int w = (v0 >> 5) + lane;
  return lane <= N ? mask[min(max(w, 0), words - 1)] : 0u;
}
template <int N>
__device__ __forceinline__ uint32_t lane_mask(uint32_t loaded, int v0, int lane) {
  const int v = v0 + lane * N, from = (v >> 5) - (v0 >> 5);
  const uint32_t a = __shfl_sync(0xffffffffu, loaded, from);
  const uint32_t b = __shfl_sync(0xffffffffu, loaded, from + 1);
  return __funnelshift_r(a, b, v & 31);
}

}  // namespace rb
