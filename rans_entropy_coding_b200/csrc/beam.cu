// beam.cu -- rans_beam_select: the best continuations of every text, over its
// beams and the vocabulary.
//
// A continuation's total is score + x - logsumexp(x) with x the row's adjusted
// logits; the order is that of totals in 64 bits, of equal ones by beam.  Within a row
// it is the order of x, which is exact (totals cannot say otherwise, only be equal), so
// rows and parts of rows can be thinned out to their best few before any sum is known;
// only between beams do the sums decide.
//
// Two launches.  The first reads the rows once.  A block takes part of a row and
// keeps, per thread, the running maximum and sum of exponentials, and in
// shared memory the tokens that may be among its best `count`: at least `count`
// threads have met a logit as large as the count-th largest of the threads'
// maxima, so nothing below that need be kept.  The second merges a text's parts.
//
// The sums: a term e^x is 2^k 2^f with k = round(x log2 e), f = x log2 e - k, log2 e in two
// parts (so f is off by no more than its two last roundings, 0.35 units of 2^-24 in the
// term; a difference x - top and its product were off by up to 11 units, all together
// where a row's body is one logit) and 2^f from the special function unit (2.45 units
// at most: measured over every float32 from -0.5 to 0.5).  k is counted from a whole
// number near the row's top.  A vector's terms add up in a tree of float32 (three
// additions of a unit each, without error where the terms are equal), all else in 64
// bits.  So a row's log sum is off by 2.8 units (1.7e-7) for a body of one logit, 5.8
// (3.5e-7) for any row; measured 1.5 at most on bodies of one to four logits, far
// less where logits differ and errors average out.
// Equal rows of a call get equal sums: a thread's tokens go by their ids, not by where a
// row starts in memory, and tokens that penalties and biases touch, which come in a
// table's order, are added as integers.
//
// Measured, 256 x 131072 bf16 in 32 texts: 34 us with the merge's 6 (memory alone 10; 31
// with the terms of rounded differences, 43 with power series of 1.1 units a term in
// place of the special function unit: the FP32 pipes then take 12 instructions a logit).
// Nothing is full: 16 instructions a logit keep issue 63% busy, the special function unit
// 42%, the ALUs 38%; warps wait at barriers (thresholds over the block in tiles 0 and 2 and at
// the end), for one another's results, and SMs for those with four blocks instead of
// three.
#include <type_traits>

#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamVecs = 4;      // vectors of 16 bytes a lane has in a tile
constexpr int kBeamList = 1024;   // tokens kept by a block
constexpr int kRanked = 256;      // of them, that are thinned out by their ranks
constexpr int kMergeThreads = 256;
constexpr int kMergeList = 512;
constexpr int kMergeItems = 4;   // candidates of a thread in registers
static_assert(RANS_MAX_CONTINUATIONS <= kBeamThreads, "a threshold needs that many maxima");

// What adjusts a call's logits: nothing, a mask alone, penalties or biases (and a mask).
enum { kPlain, kMask, kTables };
// Blocks of the first launch that an SM takes at once.  With tables two fit into its 228
// KB (66592 bytes of table, 16384 of mask bits, 8.5 KB besides); a rule that counted
// three planned half as many blocks again and ran them in a second turn (80 x 128256 f16
// under penalties: 43 us for 31; 100 x 50021: 35 for 28).  Of the others registers take
// four, of float32 three (128 x 131072: 29.4 us for 30.3 with four, which spill).
template <typename T>
constexpr int blocks_of(int adj) {
  return adj == kTables ? 2 : sizeof(T) == 4 ? 3 : 4;
}

// What a block says of its part of a row.
struct Part {
  double sum;   // of e^(x - top)
  float top;
  int32_t n;    // candidates, -1: a bad logit or parameter
};
struct Candidate {
  float x;
  int32_t token;
};

// Floats in the order of their values, as integers (-0 as 0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr float kLowest = -3.402823466e38f;
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(__dadd_rn(x, 0.0));
  return b >> 63 ? ~b : b | 1ull << 63;
}
constexpr double kLowest64 = -1.7976931348623157e308;

// The order of continuations of equal totals: the lower beam, then the larger logit,
// then the lower token.
constexpr int kTokenBits = 19, kPlaceBits = kTokenBits + 32;
static_assert(RANS_MAX_VOCAB <= 1 << kTokenBits && RANS_MAX_BEAMS < 1 << (63 - kPlaceBits),
              "places");
__device__ __forceinline__ uint64_t place_of(int beam, float x, int token) {
  return (uint64_t)beam << kPlaceBits | (uint64_t)~key_of(x) << kTokenBits | (uint64_t)token;
}

__device__ __forceinline__ int block_sum(int x, int *words) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += words[i];
  return s;
}

// A value that at least `count` of the threads' values reach, near the largest
// such, down from the largest, `most`, in steps twice as long each; -inf if fewer
// are above it.  (Not the type's lowest then: a logit may be that, too.)
template <typename F>
__device__ __forceinline__ F threshold(F mine, int count, F most, F lowest) {
  F lo = most, hi = most, d = 1;
  if (__syncthreads_count(mine >= lowest) < count) return -(F)__builtin_huge_val();
  int n = __syncthreads_count(mine >= most);
  if (n >= count) return most;
  for (;;) {
    lo = most - d;
    if (!(lo > lowest)) return lowest;
    n = __syncthreads_count(mine >= lo);
    if (n >= count) break;
    hi = lo;
    d *= 2;
  }
  for (int i = 0; i < 6 && n > count + count / 2; ++i) {
    const F mid = (lo + hi) / 2;
    const int m = __syncthreads_count(mine >= mid);
    if (m >= count) {
      lo = mid;
      n = m;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// The exact cut: a key and a place such that the items above the key, and those
// at it up to the place, are the best min(count, all), ties by place.  From `lo`
// on, which at least `count` items reach (or nothing more is below than above it).
// reach(k): how many items' keys are >= k; equal(k, p): how many are k, up to place p.
template <typename K, typename P, class Reach, class Equal>
__device__ __forceinline__ void exact_cut(int count, K lo, K most, P places, K &cut, P &last,
                                          Reach reach, Equal equal) {
  K hi = most;
  while (lo < hi) {
    const K mid = lo + (hi - lo + 1) / 2;
    if (reach(mid) >= count) lo = mid;
    else hi = mid - 1;
  }
  const int need = count - reach(lo + 1);
  P a = 0, b = places;
  while (a < b) {
    const P mid = a + (b - a) / 2;
    if (equal(lo, mid) >= need) b = mid;
    else a = mid + 1;
  }
  cut = lo;
  last = a;
}

// Two at a time.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ uint64_t both(float a) { return pair_of(a, a); }
__device__ __forceinline__ float2 halves(uint64_t x) {
  return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The larger of a vector's elements and `low`, one of its type (twice, for 16 bits).
template <typename T>
__device__ __forceinline__ uint4 at_least(const uint4 &q, uint32_t low) {
  if constexpr (sizeof(T) == 2) {
    return make_uint4(pair_most(q.x, low, T()), pair_most(q.y, low, T()),
                      pair_most(q.z, low, T()), pair_most(q.w, low, T()));
  } else {
    const float f = __uint_as_float(low);
    return make_uint4(__float_as_uint(fmaxf(__uint_as_float(q.x), f)),
                      __float_as_uint(fmaxf(__uint_as_float(q.y), f)),
                      __float_as_uint(fmaxf(__uint_as_float(q.z), f)),
                      __float_as_uint(fmaxf(__uint_as_float(q.w), f)));
  }
}

// What a thread's sum is relative to: 2^whole, or, where logits are so large (kFar) that
// x - base is exact for whatever counts, e^base.
template <typename T>
struct Reference {
  static constexpr float kFar = 4096.0f;
  static constexpr float kSlack = 32.0f;  // logits above the reference by less stay with it
  static constexpr float kDepth = 64.0f;  // those further below count as such, which no sum notices
  static constexpr double kLn2 = 0.693147180559945309417;
  float at = kNegInf, base = 0.0f, whole = 0.0f;
  // kDepth below, as logits lie in memory (about), or -inf: then below x - base instead
  uint32_t low;
  bool outside;

  __device__ __forceinline__ bool some() const { return at > kNegInf; }
  // Moves to a logit that lies too far above; what a sum is multiplied by then.
  __device__ __forceinline__ void raise(float to, float inv, double &sum) {
    if (!(to > at + kSlack)) return;
    const bool far = !(fabsf(to) < kFar);
    const float b = far ? to : 0.0f, w = far ? 0.0f : rintf(__fmul_rn(to, 0x1.715476p+0f));
    if (sum != 0.0)
      sum *= exp((double)base - (double)b + ((double)whole - (double)w) * kLn2);
    at = to;
    base = b;
    whole = w;
    // (not where the type rounds that to something else: beyond its range, by its steps
    // near 0)
    T t = float_logit<T>(__fdiv_rn(__fsub_rn(to, kDepth), inv));
    const float back = __fmul_rn(logit_float(t), inv);
    outside = far || !(back < to - 40.0f && back > to - 85.0f);
    if (outside) t = float_logit<T>(kNegInf);
    if constexpr (sizeof(T) == 2)
      low = (uint32_t)*reinterpret_cast<const uint16_t *>(&t) * 0x10001u;
    else
      low = *reinterpret_cast<const uint32_t *>(&t);
  }
  // x - base, not further below than kDepth.
  __device__ __forceinline__ uint64_t inside(uint64_t x) const {
    const float floor = __fsub_rn(__fsub_rn(at, base), kDepth);
    const float2 d = halves(add2(x, both(-base)));
    return pair_of(fmaxf(d.x, floor), fmaxf(d.y, floor));
  }
  // e^(the reference - to)
  __device__ __forceinline__ double over(float to) const {
    return exp((double)base - (double)to + (double)whole * kLn2);
  }
};

// 2^x by the special function unit.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The sum of N terms e^x relative to 2^whole.
template <int N>
__device__ __forceinline__ float vector_sum(const uint64_t (&x)[N / 2], float whole) {
  const float magic = __fsub_rn(12582912.0f, whole);  // k - whole in its low bits
  uint64_t e[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    // log2 e = 0x1.715476p+0 + 0x1.4ae0cp-26
    const uint64_t j = fma2(x[i], both(0x1.715476p+0f), both(magic));
    uint64_t f = fma2(x[i], both(0x1.715476p+0f), sub2(both(magic), j));
    f = fma2(x[i], both(0x1.4ae0cp-26f), f);
    const float2 y = halves(f);
    e[i] = pair_of(__uint_as_float(__float_as_uint(exp2_of(y.x)) + ((uint32_t)j << 23)),
                   __uint_as_float(__float_as_uint(exp2_of(y.y)) + ((uint32_t)(j >> 32) << 23)));
  }
#pragma unroll
  for (int o = N / 4; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < o; ++i) e[i] = add2(e[i], e[i + o]);
  }
  const float2 p = halves(e[0]);
  return __fadd_rn(p.x, p.y);
}
// The largest element of a vector, NaN if one is.
template <typename T>
__device__ __forceinline__ float vector_max(const uint4 &q) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t m = pair_max(pair_max(q.x, q.y, T()), pair_max(q.z, q.w, T()), T());
    float z[8];
    unpack16(make_uint4(m, 0, 0, 0), z, T());
    return max_nan(z[0], z[1]);
  } else {
    return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                   max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
}

// A vector with -inf in the places whose bit is 0.
template <typename T>
__device__ __forceinline__ uint4 keep_bits(const uint4 &q, uint32_t ok) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      constexpr uint32_t kDead = std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
      const uint32_t b = ok >> (2 * i) & 3u, m = ((b | b << 15) & 0x00010001u) * 0xffffu;
      w[i] = (w[i] & m) | (kDead & ~m);
    } else {
      w[i] = ok >> i & 1 ? w[i] : 0xff800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int ADJ>
__global__ void __launch_bounds__(kBeamThreads, blocks_of<T>(ADJ))
    beam_rows_kernel(rans_logits in, rans_adjust adj, const float *scores, int count, int parts,
                     int slice, Part *part_out, Candidate *cand_out) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int N = VecOf<T>::N;
  constexpr int kWarpTile = 32 * N * kBeamVecs;
  TouchTable &table = *reinterpret_cast<TouchTable *>(smem);
  uint32_t *ok_bits = reinterpret_cast<uint32_t *>(smem + (ADJ == kTables ? sizeof(TouchTable) : 0));
  __shared__ Candidate list[kBeamList];
  __shared__ int listed, emitted, words[kBeamWarps];
  __shared__ double sums[kBeamWarps];
  __shared__ unsigned long long whole_sums[kBeamWarps];
  __shared__ RowAdjust a;
  __shared__ float head_score;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t r = blockIdx.x / parts;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  const int lo = row.shift + (int)(blockIdx.x % parts) * slice, hi = min(lo + slice, row.end());
  Part *part = part_out + blockIdx.x;
  Candidate *out = cand_out + (int64_t)blockIdx.x * 2 * count;
  // (the merge may prepare itself meanwhile)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    // one thread reads what decides whether the row is worked on
    head_score = scores[r];
    listed = emitted = 0;
    if (ADJ) a = row_adjust(adj, r, in.vocab);
  }
  __syncthreads();
  const float inv = adj.params ? adj.params[4 * r + 3] : adj.inv_temperature;
  const bool good = inv > 0.0f && inv < __builtin_huge_valf();
  if (lo >= hi || head_score == kNegInf || !good) {
    if (tid == 0) *part = Part{0.0, kNegInf, good ? 0 : -1};
    return;
  }

  const bool touch = ADJ == kTables && a.touches();
  int table_at = -1, span = 1 << 30;
  bool dense = false;
  auto need_table = [&](int u_lo) {
    if (!ADJ || table_at == u_lo) return;
    if (touch) {
      span = fill_touch(table, a, row, u_lo, hi, dense, ok_bits, tid, kBeamThreads,
                        [] { __syncthreads(); });
    } else {
      span = min(kHashSpan, hi - u_lo);
      __syncthreads();
      fill_mask(ok_bits, a.mask, a.mask_words, row, u_lo, span, tid, kBeamThreads);
      __syncthreads();
    }
    table_at = u_lo;
  };
  // The vector of the tokens at u0, a whole number of vectors after token 0; where
  // the row starts off 16 bytes it is joined from the two that hold it.
  auto raw_at = [&](int u0, int u_hi) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (u0 < u_hi) q = load_joined(row.at0 + row.shift, row.at0 + u0, row.at0 + row.end());
    return q;
  };
  auto ok_at = [&](int u0, int u_hi) -> uint32_t {
    if (u0 >= u_hi) return 0u;
    if constexpr (ADJ) return ok_bits[(u0 - table_at) >> 5] >> ((u0 - table_at) & 31);
    else return (1u << min(row.end() - u0, N)) - 1u;
  };
  auto logits_of = [&](const uint4 &q, uint32_t ok, float (&x)[N]) {
    unpack16(q, x, T());
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = ok >> i & 1 ? __fmul_rn(x[i], inv) : kNegInf;
  };
  // walks the part, a table's tokens at a time: body(u_lo, u_hi), then touched_body()
  // where there are touched ones
  auto walk = [&](auto body, auto touched_body) {
    for (int u_lo = lo, u_hi; u_lo < hi; u_lo = u_hi) {
      need_table(u_lo);
      u_hi = span < hi - u_lo ? u_lo + span : hi;
      body(u_lo, u_hi);
      if (ADJ && touch) touched_body();
    }
  };
  auto touched = [&](auto body) {  // body(u, x)
    each_touched(table, tid, kBeamThreads, [&](int u, float z) { body(u, __fmul_rn(z, inv)); });
  };

  // mine: this thread's largest logit; ref: what its sum is relative to (the block's
  // largest so far, as far as it was asked for)
  float mine = kNegInf, cut = kNegInf;
  Reference<T> ref;
  double s = 0.0;
  float touched_top = kNegInf;
  double touched_sum = 0.0;
  auto keep = [&](int u, float x) {
    const int at = atomicAdd(&listed, 1);
    if (at < kBeamList) list[at] = Candidate{x, u - row.shift};
  };
  auto most_key = [&](float x) {  // of all threads
    const uint32_t k = __reduce_max_sync(0xffffffffu, key_of(x));
    __syncthreads();
    if (lane == 0) words[wid] = (int)k;
    __syncthreads();
    uint32_t m = 0;
    for (int i = 0; i < kBeamWarps; ++i) m = max(m, (uint32_t)words[i]);
    return m;
  };
  auto value_of = [](uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
  };

  // A warp's tile, -inf where nothing counts.  SCALED: inv is not 1.
  int round = 0;
  auto tile = [&](auto scaled, const uint4 (&q)[kBeamVecs], int u, int u_hi) {
    constexpr bool SCALED = decltype(scaled)::value;
    float m = kNegInf;
#pragma unroll
    for (int k = 0; k < kBeamVecs; ++k) {
      // compared as it lies in memory: x is monotonous in z
      m = max_nan(m, __fmul_rn(vector_max<T>(q[k]), inv));
    }
    mine = max_nan(mine, m);
    // the first tile says what to look for; tiles 2, 8, 32, ... raise it
    const bool fresh = round == 0 || ((round & 0x2aaaaaaa) == round && (round & (round - 1)) == 0);
    if (fresh) {
      const float most = value_of(most_key(mine));
      ref.raise(most, inv, s);
      cut = fmaxf(cut, threshold(mine, count, most, kLowest));
    }
    ref.raise(m, inv, s);
    if (ref.some()) {
#pragma unroll
      for (int k = 0; k < kBeamVecs; ++k) {
        float x[N];
        unpack16(at_least<T>(q[k], ref.low), x, T());
        uint64_t pairs[N / 2];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          pairs[i / 2] = pair_of(x[i], x[i + 1]);
          if constexpr (SCALED) pairs[i / 2] = mul2(pairs[i / 2], both(inv));
        }
        if (ref.outside) {
#pragma unroll
          for (int i = 0; i < N / 2; ++i) pairs[i] = ref.inside(pairs[i]);
        }
        s += (double)vector_sum<N>(pairs, ref.whole);
      }
    }
    // A warp goes through what few lanes have: perhaps among the best (ties with the cut
    // of an earlier tile are not: their tokens are higher).
    const bool keeps = fresh ? m >= cut && m > kNegInf : m > cut;
    for (uint32_t lanes = __ballot_sync(0xffffffffu, keeps); lanes != 0; lanes &= lanes - 1) {
      const int l = __ffs(lanes) - 1;
      const int k = lane / N, at = u + (l - lane) * N + 32 * N * k + lane % N;
      if (k < kBeamVecs && at < u_hi &&
          (!ADJ || ok_bits[(at - table_at) >> 5] >> ((at - table_at) & 31) & 1)) {
        const float x = __fmul_rn(logit_float(row.at0[at]), inv);
        if ((fresh ? x >= cut : x > cut) && x > kNegInf) keep(at, x);
      }
    }
  };
  walk([&](int u_lo, int u_hi) {
    constexpr int kTile = kWarpTile * kBeamWarps;
    uint4 q[kBeamVecs], next[kBeamVecs];
    const int u_first = u_lo + wid * kWarpTile + lane * N;
    auto fetch = [&](int u, int end) {  // a tile that ends at `end`
      if (row.shift == 0 && end <= u_hi) {
#pragma unroll
        for (int k = 0; k < kBeamVecs; ++k)
          next[k] = *reinterpret_cast<const uint4 *>(row.at0 + u + 32 * N * k);
      } else {
#pragma unroll
        for (int k = 0; k < kBeamVecs; ++k) next[k] = raw_at(u + 32 * N * k, u_hi);
      }
    };
    fetch(u_first, u_lo + kTile);
    for (int u = u_first, base = u_lo; base < u_hi; u += kTile, base += kTile, ++round) {
#pragma unroll
      for (int k = 0; k < kBeamVecs; ++k) q[k] = next[k];
      if (base + kTile < u_hi) fetch(u + kTile, base + 2 * kTile);
      if (ADJ || base + kTile > u_hi) {
#pragma unroll
        for (int k = 0; k < kBeamVecs; ++k)
          q[k] = keep_bits<T>(q[k], ok_at(u + 32 * N * k, u_hi));
      }
      if (inv != 1.0f) tile(std::true_type(), q, u, u_hi);
      else tile(std::false_type(), q, u, u_hi);
    }
  }, [&] {
    // their own maximum, and their sum in units of 2^-50 of it (below 2^13 of them at a
    // time)
    float m = kNegInf;
    touched([&](int u, float x) {
      m = max_nan(m, x);
      if (x >= cut && x > kNegInf) keep(u, x);
    });
    m = value_of(most_key(m));
    if (m > kNegInf) {
      unsigned long long q = 0;
      touched([&](int, float x) {
        if (x > kNegInf) q += __double2ull_rn(exp((double)x - (double)m) * 0x1p+50);
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (lane == 0) whole_sums[wid] = q;
      __syncthreads();
      q = 0;
      for (int i = 0; i < kBeamWarps; ++i) q += whole_sums[i];
      const float both = max_nan(touched_top, m);
      touched_sum = touched_sum * exp((double)touched_top - (double)both) +
                    (double)q * 0x1p-50 * exp((double)m - (double)both);
      touched_top = both;
    } else if (m != m) {
      touched_top = m;
    }
  });

  // the part's maximum and sum
  const bool bad = __syncthreads_or(!(mine < __builtin_huge_valf()) ||
                                    !(touched_top < __builtin_huge_valf()));
  if (bad) {
    if (tid == 0) *part = Part{0.0, kNegInf, -1};
    return;
  }
  const float all_top = fmaxf(value_of(most_key(mine)), touched_top);
  cut = fmaxf(cut, threshold(mine, count, all_top, kLowest));
  double sum = 0.0;
  if (ref.some()) sum = s * ref.over(all_top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sums[wid] = sum;
  int n = listed;  // (after the barriers above)
  const bool whole = n <= kBeamList;
  int above = 0;
  if (whole)
    for (int i = tid; i < n; i += kBeamThreads) above += list[i].x >= cut;
  n = block_sum(above, words);
  uint32_t key = key_of(cut);
  int last = in.vocab;
  const bool ranked = whole && n > 2 * count && listed <= kRanked;
  if (ranked) {
    // a few more than the merge has room for: their ranks
    for (int i = tid; i < listed; i += kBeamThreads) {
      const Candidate c = list[i];
      int rank = 0;
      for (int j = 0; j < listed; ++j)
        rank += list[j].x > c.x || (list[j].x == c.x && list[j].token < c.token);
      if (rank < count) out[rank] = c;
    }
    if (tid == 0) emitted = min(count, listed);
  } else if (!whole || n > 2 * count) {
    // many more (ties, mostly): exactly the best `count`
    // body(key, token) for the list, or for the part's tokens up to `place`
    auto each = [&](int place, auto body) {
      if (whole) {
        for (int i = tid; i < listed; i += kBeamThreads) body(key_of(list[i].x), list[i].token);
      } else {
        walk([&](int u_lo, int u_hi) {
          const int to = min(u_hi, place < in.vocab ? place + 1 + row.shift : u_hi);
          for (int u = u_lo + tid * N; u < to; u += kBeamThreads * N) {
            float x[N];
            logits_of(raw_at(u, u_hi), ok_at(u, u_hi), x);
#pragma unroll
            for (int i = 0; i < N; ++i) body(key_of(x[i]), u + i - row.shift);
          }
        }, [&] { touched([&](int u, float x) { body(key_of(x), u - row.shift); }); });
      }
    };
    // (the cut that was looked for is reached by `count`, or is -inf)
    exact_cut(count, key_of(cut), key_of(all_top), in.vocab, key, last, [&](uint32_t k) {
      int c = 0;
      each(in.vocab, [&](uint32_t v, int) { c += v >= k; });
      return block_sum(c, words);
    }, [&](uint32_t k, int place) {
      int c = 0;
      each(place, [&](uint32_t v, int p) { c += v == k && p <= place; });
      return block_sum(c, words);
    });
  }
  auto emit = [&](float x, int token) {
    const uint32_t v = key_of(x);
    if (x > kNegInf && (v > key || (v == key && token <= last)))
      out[atomicAdd(&emitted, 1)] = Candidate{x, token};
  };
  if (ranked) {
  } else if (whole) {
    for (int i = tid; i < listed; i += kBeamThreads) emit(list[i].x, list[i].token);
  } else {
    walk([&](int u_lo, int u_hi) {
      for (int u = u_lo + tid * N; u < u_hi; u += kBeamThreads * N) {
        float x[N];
        logits_of(raw_at(u, u_hi), ok_at(u, u_hi), x);
#pragma unroll
        for (int i = 0; i < N; ++i) emit(x[i], u + i - row.shift);
      }
    }, [&] { touched([&](int u, float x) { emit(x, u - row.shift); }); });
  }
  __syncthreads();
  if (tid == 0) {
    double all = touched_sum > 0.0 ? touched_sum * exp((double)touched_top - (double)all_top) : 0.0;
    for (int i = 0; i < kBeamWarps; ++i) all += sums[i];
    *part = Part{all, all_top, emitted};
  }
}

// One block per text.
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const float *scores, int beams, int count, int parts,
                      const Part *part_in, const Candidate *cand_in, float *out_scores,
                      int32_t *out_tokens, int32_t *out_parents, int32_t *status) {
  // score - log of the sum of e^(x - top), and top: a total is base + (x - top).  (With one
  // number for both, rows at the type's lowest value would lose the score and the sum.)
  __shared__ double base[RANS_MAX_BEAMS];
  __shared__ float tops_of[RANS_MAX_BEAMS];
  __shared__ double total[kMergeList];
  __shared__ uint64_t place[kMergeList];
  __shared__ int listed, words[kMergeThreads / 32];
  __shared__ double tops[kMergeThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t t = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) listed = 0;
  // Candidates that fit the block's registers are asked for at once, with all else.
  const int slots = 2 * count, items = beams * parts * slots;
  const int64_t first = t * beams * parts;
  const bool few = items <= kMergeItems * kMergeThreads;
  Candidate kept[kMergeItems];
  int parts_n[kMergeItems];
#pragma unroll
  for (int k = 0; k < kMergeItems; ++k) {
    const int i = tid + k * kMergeThreads;
    if (few && i < items) {
      kept[k] = cand_in[first * slots + i];
      parts_n[k] = part_in[first + i / slots].n;
    }
  }
  // a warp per beam
  for (int b = wid; b < beams; b += kMergeThreads / 32) {
    const int64_t r = t * beams + b;
    const float score = scores[r];
    float top = kNegInf;
    bool bad = !(score < __builtin_huge_valf());
    for (int p = lane; p < parts; p += 32) {
      const Part &x = part_in[r * parts + p];
      bad |= x.n < 0;
      top = fmaxf(top, x.top);
    }
    bad = __any_sync(0xffffffffu, bad) && score != kNegInf;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    double sum = 0.0;
    for (int p = lane; p < parts; p += 32) {
      const Part &x = part_in[r * parts + p];
      if (x.n >= 0 && x.top > kNegInf) sum += x.sum * exp((double)x.top - (double)top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const bool some = !bad && top > kNegInf && score > kNegInf;
      base[b] = some ? (double)score - log(sum) : -__builtin_huge_val();
      tops_of[b] = top;
      if (bad && status) report(status, RANS_ERR_RANGE, r);
    }
  }
  __syncthreads();
  // body(total, place) for all candidates of the text
  auto each = [&](auto body) {
    auto one = [&](int i, int n, const Candidate &x) {
      const int p = i / slots, b = p / parts;
      const double c = base[b];
      if (i - p * slots < n && c > -__builtin_huge_val())
        body(c + ((double)x.x - (double)tops_of[b]), place_of(b, x.x, x.token));
    };
    if (few) {
#pragma unroll
      for (int k = 0; k < kMergeItems; ++k)
        if (tid + k * kMergeThreads < items) one(tid + k * kMergeThreads, parts_n[k], kept[k]);
    } else {
      for (int i = tid; i < items; i += kMergeThreads)
        one(i, part_in[first + i / slots].n, cand_in[first * slots + i]);
    }
  };
  double best = -__builtin_huge_val();
  each([&](double v, uint64_t) { best = fmax(best, v); });
  double most = best;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) tops[wid] = most;
  __syncthreads();
  for (int i = 0; i < kMergeThreads / 32; ++i) most = fmax(most, tops[i]);
  const double cut = threshold(best, count, most, kLowest64);
  each([&](double v, uint64_t p) {
    if (v < cut) return;
    const int at = atomicAdd(&listed, 1);
    if (at < kMergeList) {
      total[at] = v;
      place[at] = p;
    }
  });
  __syncthreads();
  if (listed > kMergeList) {
    uint64_t key;
    uint64_t last = 0;
    exact_cut(count, key_of(cut), key_of(most), ~(uint64_t)0 >> 1, key, last, [&](uint64_t k) {
      int c = 0;
      each([&](double v, uint64_t) { c += key_of(v) >= k; });
      return block_sum(c, words);
    }, [&](uint64_t k, uint64_t q) {
      int c = 0;
      each([&](double v, uint64_t p) { c += key_of(v) == k && p <= q; });
      return block_sum(c, words);
    });
    __syncthreads();
    if (tid == 0) listed = 0;
    __syncthreads();
    each([&](double v, uint64_t p) {
      const uint64_t x = key_of(v);
      if (x > key || (x == key && p <= last)) {
        const int at = atomicAdd(&listed, 1);
        total[at] = v;
        place[at] = p;
      }
    });
    __syncthreads();
  }
  // each one's rank is its place in the result
  const int n = listed;
  for (int i = tid; i < n; i += kMergeThreads) {
    const double v = total[i];
    const uint64_t p = place[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += total[j] > v || (total[j] == v && place[j] < p);
    if (rank < count) {
      out_scores[t * count + rank] = (float)v;
      out_tokens[t * count + rank] = (int)(p & ((1u << kTokenBits) - 1));
      out_parents[t * count + rank] = (int)(p >> kPlaceBits);
    }
  }
  for (int i = n + tid; i < count; i += kMergeThreads) {
    out_scores[t * count + i] = kNegInf;
    out_tokens[t * count + i] = -1;
    out_parents[t * count + i] = -1;
  }
}

// Parts of a row, of so many tiles each that the blocks, as many at once as an SM
// takes, are done soonest; a block has `extra` tiles' worth of work besides (its first
// threshold, a table of touched tokens).
constexpr int kTableBytes = (int)sizeof(TouchTable) + kHashSpan / 8;  // of a block with tables
constexpr int kBlockBytes = kTableBytes + kBeamList * (int)sizeof(Candidate) + 240 + 1024;
static_assert(blocks_of<float>(kTables) * kBlockBytes <= 228 * 1024 &&
                  (blocks_of<float>(kTables) + 1) * kBlockBytes > 228 * 1024,
              "the blocks with tables that an SM takes");
struct BeamShape {
  int parts, slice;
};
constexpr int kMostParts = 64;
template <typename T>
BeamShape beam_shape(int64_t rows, int vocab, int sms, bool tables) {
  constexpr int kTile = kBeamThreads * kBeamVecs * VecOf<T>::N;
  const int tiles = (vocab + kTile - 1) / kTile, extra = tables ? 8 : 1;
  const int64_t slots = (int64_t)sms * blocks_of<T>(tables ? kTables : kPlain);
  int best = tiles;
  int64_t least = -1;
  for (int p = 1; p <= kMostParts && p <= tiles; ++p) {
    const int per = (tiles + p - 1) / p;
    const int64_t time = (rows * ((tiles + per - 1) / per) + slots - 1) / slots * (per + extra);
    if (least < 0 || time < least) {
      least = time;
      best = per;
    }
  }
  return {(tiles + best - 1) / best, best * kTile};
}
BeamShape beam_shape(int dtype, int64_t rows, int vocab, int sms, bool tables) {
  return dtype == RANS_LOGITS_F32 ? beam_shape<float>(rows, vocab, sms, tables)
                                  : beam_shape<__half>(rows, vocab, sms, tables);
}
uint64_t part_bytes(int64_t rows, int parts) {
  return ((uint64_t)rows * (uint64_t)parts * sizeof(Part) + 255) & ~255ull;
}

bool has_tables(const rans_adjust &adj) {
  return adj.history != nullptr || adj.bias_ids != nullptr;
}

template <typename T>
int launch_rows(const rans_logits &in, const rans_adjust &adj, const float *scores, int count,
                const BeamShape &sh, Part *parts, Candidate *cands, cudaStream_t st) {
  const bool tables = has_tables(adj), adjusted = tables || adj.mask;
  auto kern = tables     ? beam_rows_kernel<T, kTables>
              : adjusted ? beam_rows_kernel<T, kMask>
                         : beam_rows_kernel<T, kPlain>;
  const uint32_t smem =
      (tables ? (uint32_t)sizeof(TouchTable) : 0u) + (adjusted ? kHashSpan / 8 : 0u);
  if (smem && ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  kern<<<(unsigned)(in.rows * sh.parts), kBeamThreads, smem, st>>>(in, adj, scores, count, sh.parts,
                                                                   sh.slice, parts, cands);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

}  // namespace

uint64_t beam_workspace_bytes(int dtype, int64_t rows, int vocab, int count, int sms) {
  // (whether tables come with a call is not known here)
  const int a = beam_shape(dtype, rows, vocab, sms, false).parts;
  const int b = beam_shape(dtype, rows, vocab, sms, true).parts, parts = a > b ? a : b;
  return part_bytes(rows, parts) +
         (uint64_t)rows * (uint64_t)parts * 2 * (uint64_t)count * sizeof(Candidate);
}

int launch_beam_select(const rans_logits &in, const rans_adjust &adj, const float *scores,
                       int beams, int count, float *out_scores, int32_t *tokens,
                       int32_t *parents, void *ws, int32_t *status, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RANS_ERR_CUDA;
  const BeamShape sh = beam_shape(in.dtype, in.rows, in.vocab, num_sms(dev), has_tables(adj));
  if (in.rows > 0x7fffffff / sh.parts) return RANS_ERR_ARG;
  Part *parts = static_cast<Part *>(ws);
  Candidate *cands =
      reinterpret_cast<Candidate *>(static_cast<char *>(ws) + part_bytes(in.rows, sh.parts));
  int e;
  switch (in.dtype) {
    case RANS_LOGITS_F32: e = launch_rows<float>(in, adj, scores, count, sh, parts, cands, st); break;
    case RANS_LOGITS_F16: e = launch_rows<__half>(in, adj, scores, count, sh, parts, cands, st); break;
    default: e = launch_rows<__nv_bfloat16>(in, adj, scores, count, sh, parts, cands, st);
  }
  if (e) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(in.rows / beams));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_merge_kernel, scores, beams, count, sh.parts,
                            (const Part *)parts, (const Candidate *)cands, out_scores, tokens,
                            parents, status) == cudaSuccess
             ? RANS_OK
             : RANS_ERR_CUDA;
}

}  // namespace rb
