// logits_common.cuh -- reading rows of logits with their adjustments
// (penalties, biases, masks), shared by the kernels of logits.cu, tokens.cu
// and distill.cu.
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

// Mask bits of tokens v0 .. v0 + 31 in bits 0 .. 31 (0 off the row's ends; v0
// may be a few tokens below 0 where a row's first vector is partial).
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *mask, int words, int v0) {
  const int w = v0 >> 5;
  const uint32_t lo = w >= 0 && w < words ? mask[w] : 0u;
  const int s = v0 & 31;
  if (s <= 24) return lo >> s;  // the callers use 8 bits at most
  const uint32_t hi = w + 1 < words ? mask[w + 1] : 0u;
  return __funnelshift_r(lo, hi, s);
}

// Which tokens a row's history and biases touch, and their adjusted logits, in
// shared memory.  They are few, but spread out: handled where they are met,
// nearly every warp would stop for one in every vector (49 instructions per
// logit, measured on rows of 50,000 tokens with 300 touched).  So they are
// gathered and adjusted first, the kernels' main walks leave them out by a
// bitmap, and what they add comes from the table, a token per thread.
// Up to kTouchSpan tokens have a cell each.  A block with more of a row's
// tokens covers up to kHashSpan at once with a hash table, if the row's window
// (history and biases together) has at most kHashWindow entries; else it goes
// kTouchSpan tokens at a time.
constexpr int kHashSlots = 4096;
constexpr int kHashWindow = kHashSlots / 2;
constexpr int kHashSpan = 1 << 17;
constexpr int kTouchSpan = 8192;

struct __align__(16) TouchTable {
  union {
    struct {
      uint32_t bits[kHashSpan / 32];
      int32_t key[kHashSlots];    // place in the span, or -1
      uint32_t count[kHashSlots]; // occurrences; then the adjusted logit
      uint32_t bias[kHashSlots];  // 1 + the last entry's position in the row's list
    } hash;
    struct {
      uint32_t bits[kTouchSpan / 32];
      uint32_t count[kTouchSpan];
      uint32_t bias[kTouchSpan];
    } cells;
  };
  bool hashed;
  int u_lo, span;  // covers u in [u_lo, u_lo + span)

  __device__ __forceinline__ uint32_t *bitmap() { return hashed ? hash.bits : cells.bits; }
  // Bits of the touched ones of N tokens from u0 on (a multiple of N).
  template <int N>
  __device__ __forceinline__ uint32_t hits(int u0) {
    const int k = u0 - u_lo;
    return (bitmap()[k >> 5] >> (k & 31)) & ((1u << N) - 1u);
  }
};

__device__ __forceinline__ bool small_window(const RowAdjust &a) {
  return a.history_n + a.bias_n <= kHashWindow;
}
// Tokens that a table of the row's covers.
__device__ __forceinline__ int touch_span(const RowAdjust &a) {
  return small_window(a) ? kHashSpan : kTouchSpan;
}

__device__ __forceinline__ uint32_t hash_slot(int k) {
  return (uint32_t)k * 2654435761u >> 20;  // Fibonacci hashing to 12 bits
}
static_assert(kHashSlots == 1 << 12, "hash_slot gives 12 bits");

// body(u, its adjusted logit) for every touched token of the table, spread over
// the block's threads.
template <class Body>
__device__ __forceinline__ void each_touched(TouchTable &t, int tid, int threads, Body body) {
  if (t.hashed) {
    for (int s = tid; s < kHashSlots; s += threads)
      if (t.hash.key[s] >= 0)
        body(t.u_lo + t.hash.key[s], __uint_as_float(t.hash.count[s]));
  } else {
    for (int w = tid; w < kTouchSpan / 32; w += threads)
      for (uint32_t b = w * 32 < t.span ? t.cells.bits[w] : 0u; b != 0; b &= b - 1) {
        const int k = w * 32 + __ffs(b) - 1;
        body(t.u_lo + k, __uint_as_float(t.cells.count[k]));
      }
  }
}

// The adjusted logit of a touched token.
__device__ __forceinline__ float touched_logit(TouchTable &t, int u) {
  const int k = u - t.u_lo;
  if (!t.hashed) return __uint_as_float(t.cells.count[k]);
  uint32_t s = hash_slot(k);
  while (t.hash.key[s] != k) s = (s + 1) & (kHashSlots - 1);  // its bit is set: it is there
  return __uint_as_float(t.hash.count[s]);
}

// Fills the table for u in [u_lo, min(u_lo + touch_span, u_hi)); every thread
// of the block calls it, and a barrier ends it.  Counts come from integer
// adds, maxima and ors: what a token finds does not depend on the threads'
// order.
template <typename T>
__device__ __forceinline__ void fill_touch(TouchTable &t, const RowAdjust &a, const Row<T> &row,
                                           int u_lo, int u_hi, int tid, int threads) {
  const int span = min(touch_span(a), u_hi - u_lo);
  const bool hashed = span > kTouchSpan;
  const int64_t n = a.history_n + a.bias_n;
  auto place = [&](int64_t i) {
    const int v = i < a.history_n ? a.history[i] : a.bias_ids[i - a.history_n];
    const int k = v + row.shift - u_lo;
    return v >= 0 && v < row.vocab && k >= 0 && k < span ? k : -1;
  };
  // the adjusted logit of the token at place k
  auto adjusted = [&](int k, uint32_t count, uint32_t entry) {
    const int u = u_lo + k, v = u - row.shift;
    float z = logit_float(row.at0[u]);
    if (count > 0) {
      z = z > 0.0f ? __fdiv_rn(z, a.repetition) : __fmul_rn(z, a.repetition);
      z = __fsub_rn(z, __fadd_rn(__fmul_rn(__uint2float_rn(count), a.frequency), a.presence));
    }
    if (entry > 0) z = __fadd_rn(z, a.bias_values[entry - 1]);
    if (a.mask && !(a.mask[v >> 5] >> (v & 31) & 1)) z = kNegInf;
    return __float_as_uint(z);
  };
  // the first entry is on its way while the table is cleared
  const int first = tid < n ? place(tid) : -1;
  __syncthreads();
  if (tid == 0) {
    t.hashed = hashed;
    t.u_lo = u_lo;
    t.span = span;
  }
  uint32_t *bits = hashed ? t.hash.bits : t.cells.bits;
  for (int i = tid; i < (span + 31) / 32; i += threads) bits[i] = 0;
  if (hashed) {
    uint4 *key = reinterpret_cast<uint4 *>(t.hash.key);  // keys, then counts and biases
    for (int i = tid; i < kHashSlots / 4; i += threads)
      key[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int i = tid; i < kHashSlots / 2; i += threads)
      key[kHashSlots / 4 + i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid; i < (int)n; i += threads) {
      const int k = i == tid ? first : place(i);
      if (k < 0) continue;
      atomicOr(&bits[k >> 5], 1u << (k & 31));
      uint32_t s = hash_slot(k);
      // at most kHashWindow keys: a free slot is always found
      for (int old; (old = atomicCAS(&t.hash.key[s], -1, k)) != -1 && old != k;)
        s = (s + 1) & (kHashSlots - 1);
      if (i < a.history_n) atomicAdd(&t.hash.count[s], 1u);
      else atomicMax(&t.hash.bias[s], (uint32_t)(i - a.history_n) + 1u);
    }
    __syncthreads();
    for (int s = tid; s < kHashSlots; s += threads)
      if (t.hash.key[s] >= 0)
        t.hash.count[s] = adjusted(t.hash.key[s], t.hash.count[s], t.hash.bias[s]);
  } else {
    // only cells that are touched are ever read, so only those are cleared
    __syncthreads();
    for (int64_t i = tid; i < n; i += threads) {
      const int k = i == tid ? first : place(i);
      if (k < 0) continue;
      t.cells.count[k] = 0;
      t.cells.bias[k] = 0;
      atomicOr(&bits[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    for (int64_t i = tid; i < n; i += threads) {
      const int k = i == tid ? first : place(i);
      if (k < 0) continue;
      if (i < a.history_n) atomicAdd(&t.cells.count[k], 1u);
      else atomicMax(&t.cells.bias[k], (uint32_t)(i - a.history_n) + 1u);
    }
    __syncthreads();
    for (int w = tid; w < (span + 31) / 32; w += threads)
      for (uint32_t b = bits[w]; b != 0; b &= b - 1) {
        const int k = w * 32 + __ffs(b) - 1;
        t.cells.count[k] = adjusted(k, t.cells.count[k], t.cells.bias[k]);
      }
  }
  __syncthreads();
}

// -inf where the row's mask is 0.
template <int N>
__device__ __forceinline__ void mask_vector(float (&z)[N], const RowAdjust &a, int v0) {
  const uint32_t ok = mask_bits(a.mask, a.mask_words, v0);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (!(ok >> i & 1)) z[i] = kNegInf;
}

}  // namespace rb
