// distill.cu -- the coder's rate as a loss: distillation from a teacher's
// listed probabilities and tail, forward and backward.
//
// Write c = inv_temperature * log2(e).  The listed tokens are few: their terms
// are summed in double.  All others only enter through their own sum
//   R = sum over others of 2^(c (z - s)),   s = their largest logit,
// so that a student's small tail mass keeps its precision (1 - sum q would lose
// it).  With m the row's largest logit and Z = sum of e^(inv_t (z - m)) over all,
// the gradient of an unlisted token is 2^(c (z - s)) times one factor per row,
// inv_t (P q_t - p_t) / R: one difference, two products and one exponential, with
// no difference of close numbers but z - s, which is exact where it is small.
// (As one multiply-add, c z - c s, the rounding of c s stays in every exponent:
// past logits of 10^10, as masks have them, that is more than the exponential's
// range.)
//
// A row is walked twice, once for R and once for the gradient.  With many rows a
// block takes a row; with few, a cluster of blocks shares it and exchanges its
// maxima and sums.
// Measured, loss and gradient: 4096 x 131072 bf16 with 128 listed tokens 485 to
// 498 us (4.4 TB/s of one read and one write; 328 us at the copy's rate),
// 1001 x 50021 fp16 into rows at any alignment 63 us (31 us).  What bounds the
// long rows is DRAM: four rows of 256 KB an SM are more than L2 holds, and 55%
// of the second walk's reads leave it (480 MB read for 310 MB of rows, at
// 1184 rows), at 84% of the copy's rate with the writes.  18 instructions a
// logit keep the schedulers 63% and the special function units 50% busy; four
// blocks an SM, each with a row of its own, fill one another's waits (two
// blocks of 512 threads: 640 us; rows over clusters of 4: 760 us).  The exponent
// as a difference and a product, where one multiply-add had 492 and 62 us,
// costs 1 to 2%.
#include <cmath>

#include "cluster.cuh"
#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kStreamThreads = 256;  // walk the row
constexpr int kStreamWarps = kStreamThreads / 32;
constexpr int kListThreads = 32;     // one warp for the listed tokens meanwhile
constexpr int kDisThreads = kStreamThreads + kListThreads;
constexpr int kDisVecs = 4;
constexpr int kDisCluster = 8;
constexpr uint32_t kRingBytes = kStreamWarps * 2 * kDisVecs * 32 * 16;
constexpr double kLog2eD = 1.4426950408889634;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
// 2^(c (z - s)) of two logits; c2 and s2 hold c and -s twice.
__device__ __forceinline__ float2 exp2_pair(float a, float b, uint64_t c2, uint64_t s2) {
  uint64_t x;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(pair(a, b)), "l"(s2));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(x), "l"(c2));
  const float2 f = unpair(x);
  return make_float2(exp2_fast(f.x), exp2_fast(f.y));
}

// The largest value of a packed vector (a NaN if there is one).
__device__ __forceinline__ float vector_max(const uint4 &q, float) {
  return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                 max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
}
template <typename T>
__device__ __forceinline__ float vector_max(const uint4 &q, T) {
  const uint32_t m = pair_max(pair_max(q.x, q.y, T()), pair_max(q.z, q.w, T()), T());
  float z[8];
  unpack16(make_uint4(m, 0, 0, 0), z, T());
  return max_nan(z[0], z[1]);
}

// Per-row figures from the forward pass to the backward one (8 floats).
struct RowStats {
  float others;  // s, the unlisted tokens' largest logit
  float rest;    // inv_t (P q_t - p_t) / R, the unlisted tokens' factor
  float m_all;   // m
  float inv_z;   // 1 / Z
  float mass;    // P
  float inv_p;   // 1 / sum e^(log p - base) without a tail (0: no entry left), else 1
  float base;    // the list's largest log probability without a tail, else 0
  float pad;
};
static_assert(sizeof(RowStats) == 32, "8 floats");

__device__ __forceinline__ bool present(int v, float l, int vocab) {
  return v >= 0 && v < vocab && l != kNegInf;
}

// A chunk of the list, kEntries a lane: all its loads in flight together.
constexpr int kEntries = 4;
constexpr int kChunk = 32 * kEntries;
struct Entries {
  int v[kEntries];    // token, -1 where there is no entry
  float lp[kEntries], z[kEntries];
};
__device__ __forceinline__ void load_entries(Entries &e, const int32_t *ids, const float *lp,
                                             int from, int K, int vocab, int lane, int64_t r,
                                             int32_t *status) {
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    const int i = from + j * 32 + lane;
    e.v[j] = i < K ? ids[i] : -1;
    e.lp[j] = i < K ? lp[i] : kNegInf;
  }
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    const bool ok = present(e.v[j], e.lp[j], vocab);
    if (status && !ok && e.v[j] != -1 && e.lp[j] != kNegInf) report(status, RANS_ERR_INDEX, r);
    if (!ok) e.v[j] = -1;
  }
}
template <typename T>
__device__ __forceinline__ void load_logits(Entries &e, const T *z) {
#pragma unroll
  for (int j = 0; j < kEntries; ++j) e.z[j] = e.v[j] >= 0 ? logit_float(z[e.v[j]]) : kNegInf;
}

__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// What the listed tokens give: sums over the entries present, in double.
struct ListSums {
  double m;      // largest of their logits (0 if none is finite)
  bool some;     // one is
  double z;      // e^(inv_t (z - m))
  float base;    // what is taken off their log probabilities; p = e^(log p - base)
  double p;      // p
  double plp;    // p log p
  double pz;     // p inv_t (z - m), where p > 0
  double count;
};

// By one warp; `first` holds the list's first chunk.  Without a tail only ratios
// of the list's probabilities count, so they are taken against the largest one:
// a list far from normalised (log probabilities of +-100, say) stays in float's
// range.  (Not inlined, nor
// row_loss: the streaming warps' registers are not to pay for the double
// arithmetic of these.)
template <typename T>
__device__ __noinline__ ListSums list_sums(const Entries &first, const T *z, const int32_t *ids,
                                           const float *lp, int K, int vocab, double it,
                                           bool tail, int lane) {
  Entries e = first;
  float m = kNegInf, base = kNegInf;
  for (int from = 0; from < K; from += kChunk) {
    if (from > 0) {
      load_entries(e, ids, lp, from, K, vocab, lane, 0, nullptr);
      load_logits(e, z);
    }
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      m = fmaxf(m, e.z[j]);
      if (e.v[j] >= 0) base = fmaxf(base, e.lp[j]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    base = fmaxf(base, __shfl_xor_sync(kFull, base, o));
  }
  if (tail || base == kNegInf) base = 0.0f;
  ListSums s = {m == kNegInf ? 0.0 : (double)m, m != kNegInf, 0, base, 0, 0, 0, 0};
  for (int from = 0; from < K; from += kChunk) {
    if (K > kChunk) {
      load_entries(e, ids, lp, from, K, vocab, lane, 0, nullptr);
      load_logits(e, z);
    }
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      if (e.v[j] < 0) continue;
      const double l = (double)e.lp[j] - (double)base, d = ((double)e.z[j] - s.m) * it, p = exp(l);
      s.z += exp(d);
      s.p += p;
      s.plp += p > 0.0 || p != p ? p * l : 0.0;
      s.pz += p > 0.0 ? p * d : 0.0;
      s.count += 1.0;
    }
  }
  s.z = lanes_sum(s.z);
  s.p = lanes_sum(s.p);
  s.plp = lanes_sum(s.plp);
  s.pz = lanes_sum(s.pz);
  s.count = lanes_sum(s.count);
  return s;
}

// What the list has for the gradient.
struct ListFigures {
  float m;     // largest of its logits (-inf: none is finite)
  float z;     // e^(inv_t (z - m)), summed
  float mass, pt, norm, base;
  bool ignored;  // no entry left
};
__device__ __forceinline__ ListFigures list_figures(const ListSums &s, bool tail, int vocab) {
  const bool ignored = s.count == 0.0;
  // (a sum of p without a tail is at least 1)
  const double norm = tail ? 1.0 : (ignored ? 0.0 : 1.0 / s.p);
  const double pt = !tail || s.count >= (double)vocab ? 0.0 : fmax(0.0, 1.0 - s.p);
  return {s.some ? (float)s.m : kNegInf, (float)s.z, (float)(s.p * norm + pt), (float)pt,
          (float)norm, s.base, ignored};
}

// The row's figures from the list's and R, the sum of 2^(c (z - m_rest)) over the
// unlisted tokens, whose largest logit is m_rest (-inf: none has a finite one;
// else R is 1 at least).
// Every thread computes them for itself: in double, by one thread for all to
// wait for, this stood between the two walks for 10,000 cycles of a row's
// 100,000.  The difference P q_t - p_t is of numbers that float holds to 1e-7,
// as exact as the gradient's own terms.
__device__ __forceinline__ RowStats row_figures(const ListFigures &s, float R, float m_rest,
                                                float c, float inv_t) {
  const bool some = R > 0.0f || R != R;
  float m = fmaxf(s.m, some ? m_rest : kNegInf);
  if (m == kNegInf) m = 0.0f;
  const float rest = some ? R * exp2_fast((m_rest - m) * c) : 0.0f;
  const float top = s.m > kNegInf || s.z != s.z
                        ? s.z * exp2_fast(((s.m > kNegInf ? s.m : 0.0f) - m) * c)
                        : 0.0f;
  const float z = rest + top;
  RowStats st;
  st.others = some ? m_rest : 0.0f;
  st.rest = some && !s.ignored ? inv_t * (s.mass * (rest / z) - s.pt) / R : 0.0f;
  if (!(z > 0.0f) && !(s.ignored && z == 0.0f))  // a bad logit, or none above -inf
    st.rest = __int_as_float(0x7fffffff);
  st.m_all = m;
  st.inv_z = 1.0f / z;
  st.mass = s.mass;
  st.inv_p = s.norm;
  st.base = s.base;
  st.pad = 0.0f;
  return st;
}

// sum p (log p - log q) over the list and the tail, in double, by the listing
// warp's first thread while the others go on.
__device__ __noinline__ float row_loss(const ListSums &s, double R, float m_rest, float inv_t,
                                       bool tail, int vocab) {
  const double it = (double)inv_t;
  const bool some = R > 0.0 || R != R;
  double m = fmax(s.some ? s.m : -HUGE_VAL, some ? (double)m_rest : -HUGE_VAL);
  if (m == -HUGE_VAL) m = 0.0;
  const double rest = some ? R * exp(((double)m_rest - m) * it) : 0.0;
  const double top = s.some || s.z != s.z ? s.z * exp((s.m - m) * it) : 0.0;
  const double z = rest + top, lz = log(z);
  if (s.count == 0.0) return z == z ? 0.0f : (float)z;
  if (!(z > 0.0)) return __int_as_float(0x7fffffff);  // a bad logit, or none above -inf
  const double norm = tail ? 1.0 : 1.0 / s.p;
  const double pt = !tail || s.count >= (double)vocab ? 0.0 : fmax(0.0, 1.0 - s.p);
  double part = 0.0;
  if (s.p > 0.0 || s.p != s.p)
    part = norm * (s.plp + s.p * log(norm) - s.pz - s.p * ((s.m - m) * it - lz));
  if (pt > 0.0) {
    // the tail's logarithm from R's own: rest may be too small for a double
    const double log_rest = some ? log(R) + ((double)m_rest - m) * it : -HUGE_VAL;
    part += pt * (log(pt) - (log_rest - lz));
  }
  return (float)part;
}

// A warp's part of R.
struct Part {
  float m, r;  // largest unlisted logit; sum of 2^(c (z - m))
};

// -inf in the places of a packed vector that `hit` names.
__device__ __forceinline__ uint4 strike(uint4 q, uint32_t hit, float) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (hit >> i & 1) w[i] = 0xff800000u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 strike16(uint4 q, uint32_t hit, uint32_t dead) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = (hit >> (2 * i) & 1 ? 0xffffu : 0u) | (hit >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
    w[i] = (w[i] & ~at) | (dead & at);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 strike(uint4 q, uint32_t hit, __half) {
  return strike16(q, hit, 0xfc00fc00u);
}
__device__ __forceinline__ uint4 strike(uint4 q, uint32_t hit, __nv_bfloat16) {
  return strike16(q, hit, 0xff80ff80u);
}

// 16 bytes to shared memory under an L2 policy.
__device__ __forceinline__ void copy16(void *dst, const void *src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "l"(policy)
               : "memory");
}

enum { kForward = 1, kBackward = 2 };

// One cluster per row.  WHAT: kForward writes losses and (without kBackward)
// stats; kBackward the gradient, from stats where there is no forward pass.
template <typename T, int WHAT>
__global__ void __launch_bounds__(kDisThreads, 4)
    distill_kernel(rans_logits in, const int32_t *ids, const float *lp, int K, float inv_t,
                   int tail, float *losses, RowStats *stats, const float *grads, T *grad,
                   int64_t grad_stride, int32_t *status, int slice) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int N = VecOf<T>::N;
  constexpr int kVecRow = 32 * N, kTile = kVecRow * kDisVecs;
  __shared__ Part parts[kDisCluster * kStreamWarps];
  __shared__ ListFigures list;
  // each streaming warp's two tiles on their way; listed tokens of this
  // block's slice; the listed tokens' logits
  uint4 *ring = reinterpret_cast<uint4 *>(smem) + (threadIdx.x >> 5) * 2 * kDisVecs * 32;
  uint32_t *bits = reinterpret_cast<uint32_t *>(smem + kRingBytes);
  float *top_z = reinterpret_cast<float *>(bits + ((WHAT & kForward) ? slice / 32 : 0));
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint32_t rank = cluster_rank(), peers = cluster_size();
  const int64_t r = blockIdx.x / peers;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  const int lo = (int)rank * slice, hi = min(lo + slice, row.end());
  const bool lists = tid >= kStreamThreads;
  // (finite, so that 0 times it is 0)
  const float c = fminf((float)((double)inv_t * kLog2eD), 3.4028234663852886e38f);
  const float g = (WHAT & kBackward) ? grads[r] : 0.0f;
  ids += r * K;
  lp += r * K;
  if ((WHAT & kForward) && peers > 1) {  // waited for before the others' memory is written
    __syncwarp();
    cluster_arrive();
  }

  // Tiles reach a warp through its ring, two ahead, with no registers held
  // meanwhile; each lane copies and reads its own vectors.  (A tile that is not
  // inside the row is loaded when it is due.)
  auto inside = [&](int u) { return u >= row.shift && u + kTile <= row.end(); };
  // Four rows an SM are more than L2 holds, but half of them is behind its
  // second walk: what that has read goes first, what it will read last.  (Nearly
  // half of the second walk's reads are found there.)
  uint64_t keep, drop;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
  auto send = [&](int u, int stage, uint64_t policy) {
    if (u >= lo && u < hi && inside(u)) {
#pragma unroll
      for (int k = 0; k < kDisVecs; ++k)
        copy16(ring + (stage * kDisVecs + k) * 32 + lane,
               row.at0 + u + k * kVecRow + lane * N, policy);
    }
    cp_async_commit();
  };
  auto receive = [&](int u, int stage, uint4 (&q)[kDisVecs]) {
    cp_async_wait<1>();
    if (inside(u)) {
#pragma unroll
      for (int k = 0; k < kDisVecs; ++k) q[k] = ring[(stage * kDisVecs + k) * 32 + lane];
    } else {
#pragma unroll
      for (int k = 0; k < kDisVecs; ++k) {
        const int u0 = u + k * kVecRow + lane * N;
        if (row.whole(u0)) {
          q[k] = *reinterpret_cast<const uint4 *>(row.at0 + u0);
        } else {
          float z[N];
          row.load(u0, z, kNegInf);
          q[k] = pack16(z, T());
        }
      }
    }
    // read before the stage is written again
#pragma unroll
    for (int k = 0; k < kDisVecs; ++k)
      asm volatile("" : "+r"(q[k].x), "+r"(q[k].y), "+r"(q[k].z), "+r"(q[k].w));
  };
  constexpr int step = kStreamWarps * kTile;
  // the second walk goes backwards: what the first read last is nearest
  const int last = lo + ((hi > lo ? (hi - lo + kTile - 1) / kTile : 0) - 1 - wid) * kTile;

  RowStats st;
  ListSums sums = {};  // (the listing warp's)
  const int first = lo + wid * kTile;
  Entries e;  // (the listing warp's)
  if (lists) {
    load_entries(e, ids, lp, 0, K, in.vocab, lane, r,
                 (WHAT & kForward) && rank == 0 ? status : nullptr);
  } else if (WHAT & kForward) {
    send(first, 0, keep);
    send(first + step, 1, keep);
  }
  auto mine = [&](int v) { return v + row.shift >= lo && v + row.shift < hi; };
  // grad may be the logits' own memory: the listed ones are read before the
  // first is written
  auto read_listed = [&] {
    if (lists) load_logits(e, row.at0 + row.shift);
    if constexpr ((WHAT & kBackward) != 0)
      for (int i = kChunk + tid; i < K; i += kDisThreads)
        if (present(ids[i], lp[i], in.vocab) && mine(ids[i]))
          top_z[i] = logit_float(row.at0[row.shift + ids[i]]);
  };
  if constexpr ((WHAT & kForward) != 0) {
    for (int i = tid; i < slice / 32; i += kDisThreads) bits[i] = 0;
    __syncthreads();
    auto mark = [&](int v) {
      const int k = v + row.shift - lo;
      if (v < 0 || k < 0 || k >= hi - lo) return;
      if (atomicOr(&bits[k >> 5], 1u << (k & 31)) >> (k & 31) & 1)
        report(status, RANS_ERR_INDEX, r);  // listed twice
    };
    if (lists) {
#pragma unroll
      for (int j = 0; j < kEntries; ++j) mark(e.v[j]);
    }
    for (int i = kChunk + tid; i < K; i += kDisThreads) {
      const int v = ids[i];
      if (present(v, lp[i], in.vocab)) mark(v);
      else if (rank == 0 && v != -1 && lp[i] != kNegInf) report(status, RANS_ERR_INDEX, r);
    }
    __syncthreads();
    read_listed();
    if (lists) {
      sums = list_sums(e, row.at0 + row.shift, ids, lp, K, in.vocab, (double)inv_t,
                       tail != 0, lane);
      if (lane == 0) list = list_figures(sums, tail != 0, in.vocab);
    } else {
      // R, against each lane's running maximum
      float m = kNegInf;
      uint64_t s2 = 0;  // two sums
      const uint64_t c2 = pair(c, c);
      for (int u = first, stage = 0; u < hi; u += step, stage ^= 1) {
        uint4 q[kDisVecs];
        uint32_t word[kDisVecs];
        receive(u, stage, q);
        send(u + 2 * step, stage, keep);
        // (a tile's bits lie inside the slice's, which is a whole number of tiles)
#pragma unroll
        for (int k = 0; k < kDisVecs; ++k)
          word[k] = bits[(u - lo + k * kVecRow + lane * N) >> 5];
#pragma unroll
        for (int k = 0; k < kDisVecs; ++k) {
          const uint32_t hit = word[k] >> (lane * N & 31) & ((1u << N) - 1u);
          if (hit) q[k] = strike(q[k], hit, T());
        }
        float top = vector_max(q[0], T());
#pragma unroll
        for (int k = 1; k < kDisVecs; ++k) top = max_nan(top, vector_max(q[k], T()));
        if (!(top <= m)) {
          // (a NaN stays one, and makes all that follows NaN)
          if (m != kNegInf) {
            const float f = exp2_fast((m - top) * c);
            const float2 s = unpair(s2);
            s2 = pair(s.x * f, s.y * f);
          }
          m = top;
        }
        const float at = m == kNegInf ? 0.0f : -m;
        const uint64_t at2 = pair(at, at);
#pragma unroll
        for (int k = 0; k < kDisVecs; ++k) {
          float z[N];
          unpack16(q[k], z, T());
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float2 e = exp2_pair(z[i], z[i + 1], c2, at2);
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(s2) : "l"(s2), "l"(pair(e.x, e.y)));
          }
        }
      }
      float s = unpair(s2).x + unpair(s2).y;
      if constexpr ((WHAT & kBackward) != 0) {  // the second walk's first tiles
        send(last, 0, drop);
        send(last - step, 1, drop);
      }
      float w = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w = max_nan(w, __shfl_xor_sync(kFull, w, o));
      if (m != kNegInf) s *= exp2_fast((m - w) * c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      if (peers > 1) cluster_wait();
      if (lane < (int)peers) {
        const uint32_t at = peer_address(&parts[rank * kStreamWarps + wid], lane);
        peer_store(at, __float_as_uint(w));
        peer_store(at + 4, __float_as_uint(s));
      }
    }
    if (peers > 1) {
      if (lists) cluster_wait();
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    // the parts joined, by every warp alike
    float m_rest = kNegInf;
    for (int i = lane; i < (int)peers * kStreamWarps; i += 32)
      m_rest = max_nan(m_rest, parts[i].m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m_rest = max_nan(m_rest, __shfl_xor_sync(kFull, m_rest, o));
    float R = 0.0f;
    for (int i = lane; i < (int)peers * kStreamWarps; i += 32) {
      const Part p = parts[i];
      R += p.m == kNegInf ? p.r : p.r * exp2_fast((p.m - m_rest) * c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) R += __shfl_xor_sync(kFull, R, o);
    st = row_figures(list, R, m_rest, c, inv_t);
    if (rank == 0 && tid == kStreamThreads) {
      if constexpr (WHAT == kForward) stats[r] = st;
      losses[r] = row_loss(sums, (double)R, m_rest, inv_t, tail != 0, in.vocab);
    }
    if constexpr (WHAT == kForward) return;
  } else {
    st = stats[r];
    read_listed();
    __syncthreads();
  }

  if constexpr ((WHAT & kBackward) != 0) {
    T *o = grad + r * grad_stride - row.shift;
    if (!lists) {
      const float factor = st.rest * g;
      const uint64_t c2 = pair(c, c), at2 = pair(-st.others, -st.others);
      const uint64_t factor2 = pair(factor, factor);
      if constexpr (WHAT == kBackward) {
        send(last, 0, drop);
        send(last - step, 1, drop);
      }
      for (int u = last, stage = 0; u >= lo; u -= step, stage ^= 1) {
        uint4 q[kDisVecs];
        receive(u, stage, q);
        send(u - 2 * step, stage, drop);
#pragma unroll
        for (int k = 0; k < kDisVecs; ++k) {
          float z[N];
          unpack16(q[k], z, T());
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float2 e = exp2_pair(z[i], z[i + 1], c2, at2);
            uint64_t x;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(pair(e.x, e.y)), "l"(factor2));
            const float2 f = unpair(x);
            z[i] = f.x;
            z[i + 1] = f.y;
          }
          q[k] = pack16(z, T());
        }
        store_tile<true>(o, u, q, inside(u), row.shift, hi);
      }
    }
    __syncthreads();  // the listed tokens' gradients go over what stands there
    auto write = [&](int v, float l, float z) {
      const float q = expf((z - st.m_all) * inv_t) * st.inv_z;
      const float p = expf(l - st.base) * st.inv_p;
      o[row.shift + v] = float_logit<T>((st.mass * q - p) * inv_t * g);
    };
    if (lists) {
#pragma unroll
      for (int j = 0; j < kEntries; ++j)
        if (e.v[j] >= 0 && mine(e.v[j])) write(e.v[j], e.lp[j], e.z[j]);
    }
    for (int i = kChunk + tid; i < K; i += kDisThreads)
      if (present(ids[i], lp[i], in.vocab) && mine(ids[i])) write(ids[i], lp[i], top_z[i]);
  }
}

template <typename T, int WHAT>
int launch_t(const rans_logits &in, const int32_t *ids, const float *lp, int K, float inv_t,
             int tail, float *losses, float *stats, const float *grads, void *grad,
             int64_t stride, int32_t *status, cudaStream_t st) {
  auto kern = distill_kernel<T, WHAT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RANS_ERR_CUDA;
  constexpr int kTile = 32 * VecOf<T>::N * kDisVecs;
  const int tiles = (in.vocab + VecOf<T>::N - 1 + kTile - 1) / kTile;
  // blocks per row: one, while the rows alone fill the SMs (four blocks each);
  // else as many as still leave every warp a tile
  int peers = 1;
  while (peers < kDisCluster && in.rows * peers * 2 <= 4 * num_sms(dev) &&
         tiles >= peers * 2 * kStreamWarps)
    peers *= 2;
  const int slice = (tiles + peers - 1) / peers * kTile;
  const uint32_t smem = kRingBytes + ((WHAT & kForward) ? (uint32_t)slice / 8u : 0u) +
                        ((WHAT & kBackward) ? 4u * (uint32_t)K : 0u);
  if (smem && ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  if (in.rows > 0x7fffffff / peers) return RANS_ERR_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(in.rows * peers));
  cfg.blockDim = dim3(kDisThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)peers;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, in, ids, lp, K, inv_t, tail, losses,
                            reinterpret_cast<RowStats *>(stats), grads, static_cast<T *>(grad),
                            stride, status, slice) == cudaSuccess
             ? RANS_OK
             : RANS_ERR_CUDA;
}

template <int WHAT>
int launch(const rans_logits &in, const int32_t *ids, const float *lp, int K, float inv_t,
           int tail, float *losses, float *stats, const float *grads, void *grad, int64_t stride,
           int32_t *status, cudaStream_t st) {
  switch (in.dtype) {
    case RANS_LOGITS_F32:
      return launch_t<float, WHAT>(in, ids, lp, K, inv_t, tail, losses, stats, grads, grad,
                                   stride, status, st);
    case RANS_LOGITS_F16:
      return launch_t<__half, WHAT>(in, ids, lp, K, inv_t, tail, losses, stats, grads, grad,
                                    stride, status, st);
    default:
      return launch_t<__nv_bfloat16, WHAT>(in, ids, lp, K, inv_t, tail, losses, stats, grads,
                                           grad, stride, status, st);
  }
}

}  // namespace

int launch_distill_forward(const rans_logits &in, const int32_t *ids, const float *lp, int K,
                           float inv_t, int tail, float *losses, float *stats, int32_t *status,
                           cudaStream_t st) {
  return launch<kForward>(in, ids, lp, K, inv_t, tail, losses, stats, nullptr, nullptr, 0,
                          status, st);
}

int launch_distill_backward(const rans_logits &in, const int32_t *ids, const float *lp, int K,
                            float inv_t, const float *stats, const float *grads, void *grad,
                            int64_t stride, cudaStream_t st) {
  return launch<kBackward>(in, ids, lp, K, inv_t, 0, nullptr, const_cast<float *>(stats), grads,
                           grad, stride, nullptr, st);
}

int launch_distill(const rans_logits &in, const int32_t *ids, const float *lp, int K,
                   float inv_t, int tail, const float *grads, float *losses, void *grad,
                   int64_t stride, int32_t *status, cudaStream_t st) {
  return launch<kForward | kBackward>(in, ids, lp, K, inv_t, tail, losses, nullptr, grads, grad,
                                      stride, status, st);
}

}  // namespace rb
