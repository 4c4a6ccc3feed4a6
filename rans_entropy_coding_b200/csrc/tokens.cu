// tokens.cu -- coding tokens under a model's logits: the intervals of given
// tokens (encoder side), one decoding step for a batch of streams, and the
// streams themselves.
//
// The weight of a token is an integer computed from its logit and the row's
// maximum by float32 operations that are each rounded on their own, so every
// kernel (and any other IEEE machine) gets the same one; all sums are of
// integers, so neither the split of a row over threads nor the order of
// additions can change an interval.
#include <type_traits>

#include "cluster.cuh"
#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr uint32_t kTokPrec = RANS_TOKEN_PRECISION;
constexpr uint32_t kTokTotal = 1u << kTokPrec;
// Sums of weights stay below 2^19 * 2^21 = 2^40 and their products with
// 2^24 - N below 2^64.
static_assert(RANS_MAX_VOCAB <= (1 << 19), "weights and their products fit 64 bits");

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLowest = -64.0f;
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
constexpr float kUnit = 8388608.0f;    // 2^23
constexpr float kScaleW = 2097152.0f;  // 2^21, folded into the polynomial (exact)
constexpr float kC1 = 0x1.62f5fap-1f * kScaleW;
constexpr float kC2 = 0x1.f00c4ep-3f * kScaleW;
constexpr float kC3 = 0x1.c2a218p-5f * kScaleW;

// w = rint(2^21 p(f) 2^k): 2^21 p(f) gets k added to its exponent (k sits in
// the low bits of d + 1.5 * 2^23) and is rounded by adding 2^23.
// z = -inf gives 0 (d is clamped, also from NaN).
__device__ __forceinline__ uint32_t token_weight(float z, float scale, float ymax) {
  const float d = fmaxf(__fsub_rn(__fmul_rn(z, scale), ymax), kLowest);
  const float t = __fadd_rn(d, kRound);
  const float f = __fsub_rn(d, __fsub_rn(t, kRound));
  float p = __fadd_rn(__fmul_rn(f, kC3), kC2);
  p = __fadd_rn(__fmul_rn(p, f), kC1);
  p = __fadd_rn(__fmul_rn(p, f), kScaleW);
  const float q = __uint_as_float(__float_as_uint(p) + (__float_as_uint(t) << 23));
  return __float_as_uint(__fadd_rn(q, kUnit)) - __float_as_uint(kUnit);
}

// The factor and the reference of a row's weights from its largest adjusted
// logit.  A row whose alive tokens all overflow to -inf weighs them the same:
// with factor 0 they get d = 0, and dead ones (-inf * 0) NaN, hence -64.
struct RowScale {
  float scale, ymax;
  int error;  // RANS_OK, ERR_RANGE (bad logit) or ERR_ZERO_FREQ (no token alive)
};
__device__ __forceinline__ RowScale row_scale(float zmax, float inv_temperature) {
  RowScale s;
  s.scale = __fmul_rn(kLog2e, inv_temperature);
  s.ymax = __fmul_rn(zmax, s.scale);
  s.error = RANS_OK;
  if (!(s.scale > 0.0f && s.scale < __builtin_huge_valf())) {
    s.error = RANS_ERR_RANGE;  // (per-row parameters are not known to the host)
  } else if (zmax == kNegInf) {
    s.error = RANS_ERR_ZERO_FREQ;
  } else if (!(s.ymax < __builtin_huge_valf())) {  // NaN or +inf
    s.error = RANS_ERR_RANGE;
  } else if (s.ymax == kNegInf) {
    s.scale = 0.0f;
    s.ymax = 0.0f;
  }
  return s;
}

// Start of a token with weight sum c and r alive tokens below it.
__device__ __forceinline__ uint32_t interval_start(uint64_t c, uint32_t r, uint64_t total,
                                                   uint32_t alive) {
  return (uint32_t)(c * (uint64_t)(kTokTotal - alive) / total) + r;
}

// Whether that start is at most `slot`, without the division:
// floor(c M / W) <= s - r  <=>  c M < (s - r + 1) W, and always when s - r >= M
// (c <= W), which also keeps the right side below 2^64.
__device__ __forceinline__ bool starts_by(uint64_t c, uint32_t r, uint64_t total, uint32_t alive,
                                          uint32_t slot) {
  const uint32_t room = kTokTotal - alive;
  if (r > slot) return false;
  const uint32_t s = slot - r;
  return s >= room || c * (uint64_t)room < (uint64_t)(s + 1) * total;
}

// ------------------------------------------------------------------ rows --
// A row is shared by a cluster of 1 to kMaxCluster blocks, which exchange its
// maximum and then its sums through each other's shared memory.  Weights are
// relative to the maximum, so the row is walked twice; the second walk finds
// it in L2 (or L1).  The format's roundings cost more than the memory: 12
// operations of the FP32 pipes and 15 instructions per logit.
// Measured: 4096 x 131072 bf16 350 us (one read of the rows 164 us, the FP32
// pipes 176 us, the instructions' issue 216 us); a decoding step of 256 such
// rows 41 us (two rows on most SMs), of one row 10 us, most of it launch and two
// exchanges of 1 us.  Four blocks of 256 threads an SM instead of two of 512
// took 398 us and 43 us; a first form that held a row in registers over
// clusters of 8, 900 us and 108 us.
// A warp takes "tiles" of 32 lanes x row_vecs vectors of 16 bytes, lane after
// lane and vector row after vector row, so that a tile is a run of consecutive
// tokens whose sums a decoding row keeps.
// (Four vectors a lane; two where a row has tables or a mask, whose blocks have
// few tiles each: 48 x 50021 f32 21 us against 23, 777 x 50021 fp16 the same;
// without, 4096 x 131072 bf16 takes 425 us with two, 366 with four, 412 with
// eight.)
__host__ __device__ constexpr int row_vecs(bool adjusted) { return adjusted ? 2 : 4; }
constexpr int kRowThreads = 512;  // most threads of a block
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxCluster = 16;

struct Sums {
  uint64_t w;
  uint32_t n;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.w + b.w, a.n + b.n}; }

__device__ __forceinline__ Sums warp_total(Sums v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.w += __shfl_xor_sync(kFull, v.w, o);
  v.n = __reduce_add_sync(kFull, v.n);
  return v;
}
// Sums of this lane and the ones below it.
__device__ __forceinline__ Sums warp_scan(Sums v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t w = __shfl_up_sync(kFull, v.w, o);
    const uint32_t n = __shfl_up_sync(kFull, v.n, o);
    if (lane >= o) v = v + Sums{w, n};
  }
  return v;
}

// A warp's sums on their way to another block.
struct WarpSums {
  uint64_t w, below_w;  // weights of all its tokens; of those below the coded one
  uint32_t n, below_n;  // alive tokens
};

__device__ __forceinline__ float warp_max_nan(float x) {
  float y;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Running extremes of raw vectors, in the type they come in.
template <typename T>
struct Extremes {
  uint32_t top = sizeof(T) == 2 ? (std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u)
                                : 0xff800000u;
  uint32_t low = top & 0x7fff7fffu;
  __device__ __forceinline__ void take(const uint4 &q) {
    if constexpr (sizeof(T) == 2) {
      top = pair_max(top, pair_max(pair_max(q.x, q.y, T()), pair_max(q.z, q.w, T()), T()), T());
      low = pair_min(low, pair_min(pair_min(q.x, q.y, T()), pair_min(q.z, q.w, T()), T()), T());
    } else {
      float z[4];
      unpack16(q, z, T());
      float a = __uint_as_float(top), b = __uint_as_float(low);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a = max_nan(a, z[i]);
        b = fminf(b, z[i]);
      }
      top = __float_as_uint(a);
      low = __float_as_uint(b);
    }
  }
  __device__ __forceinline__ void take_low(const uint4 &q) {
    if constexpr (sizeof(T) == 2) {
      low = pair_min(low, pair_min(pair_min(q.x, q.y, T()), pair_min(q.z, q.w, T()), T()), T());
    } else {
      float z[4];
      unpack16(q, z, T());
#pragma unroll
      for (int i = 0; i < 4; ++i) low = __float_as_uint(fminf(__uint_as_float(low), z[i]));
    }
  }
  __device__ __forceinline__ static float2 both(uint32_t x) {
    if constexpr (sizeof(T) == 2) {
      float z[8];
      unpack16(make_uint4(x, 0, 0, 0), z, T());
      return make_float2(z[0], z[1]);
    } else {
      return make_float2(__uint_as_float(x), __uint_as_float(x));
    }
  }
  __device__ __forceinline__ float largest() const {
    const float2 f = both(top);
    return max_nan(f.x, f.y);
  }
  __device__ __forceinline__ float smallest() const {
    const float2 f = both(low);
    return fminf(f.x, f.y);
  }
};

// Two weights without the clamp (d >= -64 is the caller's to know), each with
// the bits of 2^23 still on top.  A product is written as a * b + zero2, where
// zero2 holds two -0 that the compiler does not know: it makes a packed product
// and the packed sum behind it (an explicit .rn on both, a literal -0, or
// -fmad=false notwithstanding) into one multiply-add, and half of all results
// then differ from the two roundings of the format.
__device__ __forceinline__ uint2 raw_weights(float a, float b, uint64_t scale2, uint64_t ymax2,
                                             uint64_t zero2) {
  uint64_t z, d, t, k, f, p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(a), "f"(b));
  auto both = [](float c) {
    return (uint64_t)__float_as_uint(c) << 32 | __float_as_uint(c);
  };
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(z), "l"(scale2), "l"(zero2));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(d), "l"(ymax2));  // ymax2 holds -ymax
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(d), "l"(both(kRound)));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(k) : "l"(t), "l"(both(-kRound)));
  // f = d - k is exact, so this product and sum round as the difference does
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(f) : "l"(k), "l"(both(-1.0f)), "l"(d));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(f), "l"(both(kC3)), "l"(zero2));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(p), "l"(both(kC2)));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(p), "l"(f), "l"(zero2));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(p), "l"(both(kC1)));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(p), "l"(f), "l"(zero2));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(p), "l"(both(kScaleW)));
  const uint32_t lo = (uint32_t)p + ((uint32_t)t << 23);
  const uint32_t hi = (uint32_t)(p >> 32) + ((uint32_t)(t >> 32) << 23);
  p = (uint64_t)hi << 32 | lo;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(p), "l"(both(kUnit)));
  return make_uint2((uint32_t)p, (uint32_t)(p >> 32));
}

// Where a decoding row's symbol comes from.
struct Coded {
  const uint8_t *in;
  uint64_t in_bytes;
  const uint64_t *offsets;
  int64_t S;
  const int32_t *stream_ids;
  const uint64_t *states_in;
  uint64_t *states_out;
  int32_t *tokens;
};

// The streams' side of a decoding row: a token whose interval is [s, s + f).
__device__ __forceinline__ void take_token(const Coded &cd, int64_t r, int64_t stream, uint64_t x,
                                           uint64_t taken, int token, uint32_t s, uint32_t f,
                                           bool refill_ok, uint32_t refill_word,
                                           int32_t *status) {
  uint64_t y = (uint64_t)f * (x >> kTokPrec) + (x & (kTokTotal - 1)) - s;
  uint64_t used = taken;
  if (y < kL) {
    if (refill_ok) {
      y = y << 32 | refill_word;
      used = taken + 1;
    } else {
      report(status, RANS_ERR_CORRUPT, stream);
      token = -1;
      y = x;
    }
  }
  cd.tokens[r] = token;
  cd.states_out[2 * stream] = y;
  cd.states_out[2 * stream + 1] = used;
}

// One cluster per row.  ADJ: with penalties, biases or a mask.
template <typename T, bool DECODE, bool ADJ>
__global__ void __launch_bounds__(kRowThreads, 2)
    token_rows_kernel(rans_logits in, rans_adjust adj, const int32_t *tokens, uint32_t *starts,
                      uint32_t *freqs, Coded cd, int32_t *status, int slice, uint64_t zero2) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int N = VecOf<T>::N;
  constexpr int kTileVecs = row_vecs(ADJ);
  constexpr int kVecRow = 32 * N;                // tokens of a warp's vectors
  constexpr int kTile = kVecRow * kTileVecs;
  TouchTable &table = *reinterpret_cast<TouchTable *>(smem);
  // bits of the tokens that the mask leaves and nothing touches
  uint32_t *ok_bits = reinterpret_cast<uint32_t *>(smem + (ADJ ? sizeof(TouchTable) : 0));
  uint2 *tile_sums = reinterpret_cast<uint2 *>(ok_bits + (ADJ ? kHashSpan / 32 : 0));
  __shared__ float peer_max[kMaxCluster * kRowWarps];
  __shared__ WarpSums peer_sums[kMaxCluster * kRowWarps];
  __shared__ uint32_t own_weight;
  __shared__ int found_tile;
  __shared__ Sums found_base, found_all;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  const uint32_t rank = cluster_rank(), peers = cluster_size();
  const int64_t r = blockIdx.x / peers;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);

  // One thread reads what decides whether the row is worked on: should another
  // call be writing it meanwhile, a block's threads still agree.
  __shared__ int64_t head_stream;
  __shared__ uint64_t head_state, head_taken;
  __shared__ int head_target;
  __shared__ RowAdjust a;
  if (ADJ && tid == (warps > 1 ? 32 : 0)) a = row_adjust(adj, r, in.vocab);
  // each warp's first tile comes nearer while the row's particulars are read
  const int lo = (int)rank * slice, hi = min(lo + slice, row.end());
#pragma unroll
  for (int k = 0; k < kTileVecs; ++k) {
    const int u0 = lo + wid * kTile + k * kVecRow + lane * N;
    if (u0 >= row.shift && u0 < hi)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row.at0 + u0));
  }
  if (tid == 0) {
    if constexpr (DECODE) {
      head_stream = cd.stream_ids ? (int64_t)cd.stream_ids[r] : r;
      const bool known = head_stream >= 0 && head_stream < cd.S;
      head_state = known ? cd.states_in[2 * head_stream] : 0;
      head_taken = known ? cd.states_in[2 * head_stream + 1] : 0;
    } else {
      head_target = tokens[r];
    }
  }
  __syncthreads();
  const int64_t stream = DECODE ? head_stream : r;
  const uint64_t x = DECODE ? head_state : 0, taken = DECODE ? head_taken : 0;
  const int target = DECODE ? -1 : head_target;
  // A block of a cluster may only leave when the others write to it no more, so
  // one that has nothing to do still meets their `phases` barriers.
  auto leave = [&](int phases) {
    if (peers == 1) return;
    for (int i = 0; i < phases; ++i) {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
  };
  auto refuse = [&](int phases, int code, int64_t detail, bool state) {
    if (rank == 0 && tid == 0) {
      report(status, code, detail);
      if constexpr (DECODE) {
        cd.tokens[r] = -1;
        if (state) {
          cd.states_out[2 * stream] = x;
          cd.states_out[2 * stream + 1] = taken;
        }
      } else {
        starts[r] = 0;
        freqs[r] = 0;
      }
    }
    leave(phases);
  };
  if constexpr (DECODE) {
    if (stream == -1) return leave(3);
    int bad = stream < 0 || stream >= cd.S;
    if (!bad && cd.stream_ids) {
      for (int64_t i = tid; i < in.rows; i += threads)
        bad |= i != r && cd.stream_ids[i] == (int32_t)stream;
      bad = __syncthreads_or(bad);
    }
    if (bad) return refuse(3, RANS_ERR_INDEX, r, false);
    if (x < kL || x >> 63) return refuse(3, RANS_ERR_CORRUPT, stream, true);
  } else {
    if (target == -1) return leave(3);
    if (target < 0 || target >= in.vocab) return refuse(3, RANS_ERR_INDEX, r, false);
  }
  // the word that the stream would go on with, read long before it is needed
  __shared__ uint32_t refill_word;
  __shared__ bool refill_ok;
  if (DECODE && tid == threads - 1) {
    const uint64_t off = cd.offsets[stream], lim = cd.offsets[stream + 1];
    refill_ok = !(off & 3) && off <= lim && lim <= cd.in_bytes && taken < (lim - off) / 4;
    if (refill_ok) refill_word = reinterpret_cast<const uint32_t *>(cd.in)[off / 4 + taken];
  }
  // a block's shared memory may be written by others once it runs: waited for
  // below, after the first walk
  if (peers > 1) {
    __syncwarp();
    cluster_arrive();
  }

  const bool touch = ADJ && a.touches();
  if (DECODE && ADJ && touch)  // added to after the first walk's barrier
    for (int i = tid; i < slice / kTile; i += threads) tile_sums[i] = make_uint2(0, 0);
  int table_at = -1, span = 1 << 30;  // where the table starts, its tokens
  bool dense = false;
  auto need_table = [&](int u_lo) {
    if (!ADJ || table_at == u_lo) return;
    if (touch) {
      span = fill_touch(table, a, row, u_lo, hi, dense, ok_bits, tid, threads,
                        [] { __syncthreads(); });
    } else {
      span = min(kHashSpan, hi - u_lo);
      __syncthreads();
      fill_mask(ok_bits, a.mask, a.mask_words, row, u_lo, span, tid, threads);
      __syncthreads();
    }
    table_at = u_lo;
  };
  // walks this block's tiles, body(tile's first u, its number), and the touched
  // tokens of its tables, which the tiles leave out: touched_body(u, logit)
  auto walk = [&](auto body, auto touched_body) {
    for (int u_lo = lo, u_hi; u_lo < hi; u_lo = u_hi) {
      need_table(u_lo);
      u_hi = span < hi - u_lo ? u_lo + span : hi;
      for (int u = u_lo + wid * kTile; u < u_hi; u += warps * kTile) body(u, (u - lo) / kTile);
      if (ADJ && touch) each_touched(table, tid, threads, touched_body);
    }
  };
  // A tile is loaded at once, with the bits of its tokens that count (`some`:
  // not all of them do).  Places off the row's ends read 0.
  auto inside = [&](int u) { return u >= row.shift && u + kTile <= row.end(); };
  auto load_tile = [&](int u, uint4 (&q)[kTileVecs], uint32_t (&ok)[kTileVecs]) -> bool {
    const bool edge = !inside(u);
    if (edge) {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k) {
        const int u0 = u + k * kVecRow + lane * N;
        q[k] = make_uint4(0, 0, 0, 0);
        if (row.whole(u0)) {
          q[k] = *reinterpret_cast<const uint4 *>(row.at0 + u0);
        } else if (u0 < row.end()) {
          float z[N];
          row.load(u0, z, 0.0f);
          q[k] = pack16(z, T());
        }
        const int from = min(max(row.shift - u0, 0), N), to = min(max(row.end() - u0, 0), N);
        ok[k] = (1u << to) - (1u << from);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k)
        q[k] = *reinterpret_cast<const uint4 *>(row.at0 + u + k * kVecRow + lane * N);
    }
    if constexpr (ADJ) {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k) {
        const int at = u + k * kVecRow + lane * N - table_at;
        const uint32_t b = at < span ? ok_bits[at >> 5] >> (at & 31) & ((1u << N) - 1u) : 0u;
        ok[k] = b;
      }
    }
    return ADJ || edge;
  };
  // Adjusted logits of this lane's vector at u0; those of touched tokens read
  // -inf unless asked for.  (For what is done once per row.)
  auto fetch = [&](int u0, float (&z)[N], bool all) {
    row.load(u0, z, kNegInf);
    if constexpr (ADJ) {
      const int at = u0 - table_at;
      const uint32_t b = at < span ? ok_bits[at >> 5] >> (at & 31) : 0u;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(b >> i & 1)) z[i] = all && touch ? touched_logit(table, u0 + i) : kNegInf;
    }
  };

  // First walk: the maximum of the tokens that count, and the least logit of
  // all in the tiles (which only has to be a bound).
  float m = kNegInf;
  Extremes<T> ends;
  walk([&](int u, int) {
    uint4 q[kTileVecs];
    uint32_t ok[kTileVecs];
    if (!load_tile(u, q, ok)) {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k) ends.take(q[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k) {
        ends.take_low(q[k]);
        float z[N];
        unpack16(q[k], z, T());
#pragma unroll
        for (int i = 0; i < N; ++i) m = max_nan(m, ok[k] >> i & 1 ? z[i] : kNegInf);
      }
    }
  }, [&](int, float z) { m = max_nan(m, z); });
  const float least = ends.smallest();
  m = max_nan(m, ends.largest());
  m = warp_max_nan(m);
  if (tid == 0) own_weight = 0xffffffffu;
  if (peers > 1) {
    cluster_wait();
    if (lane < (int)peers)
      peer_store(peer_address(&peer_max[rank * warps + wid], lane), __float_as_uint(m));
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  } else {
    if (lane == 0) peer_max[wid] = m;
    __syncthreads();
  }
  m = kNegInf;
  for (int i = lane; i < (int)peers * warps; i += 32) m = max_nan(m, peer_max[i]);
  m = warp_max_nan(m);
  const RowScale rs =
      row_scale(m, adj.params ? adj.params[4 * r + 3] : adj.inv_temperature);
  if (rs.error != RANS_OK) return refuse(1, rs.error, r, true);

  // Second walk: the weights.  Where a warp's smallest logit needs no clamp,
  // the only dead tokens are those that do not count, and the weights go two at
  // a time; such a token then takes a logit whose d is -40, hence weight 0
  // (which wants a maximum that 40 can be told from, and a factor).
  const int u_target = row.shift + target;
  const float dead = (rs.ymax - 40.0f) / rs.scale;
  const bool plain = __all_sync(
      kFull, __fsub_rn(__fmul_rn(least, rs.scale), rs.ymax) >= kLowest && least > kNegInf &&
                 fabsf(rs.ymax) < 65536.0f && fabsf(dead) < 1e30f);
  const uint64_t scale2 = (uint64_t)__float_as_uint(rs.scale) << 32 | __float_as_uint(rs.scale);
  const uint64_t ymax2 =
      (uint64_t)__float_as_uint(-rs.ymax) << 32 | __float_as_uint(-rs.ymax);
  WarpSums s = {0, 0, 0, 0};
  walk([&](int u, int tile) {
    // a lane's weights of a tile sum to at most 2^26, a tile's to 2^31
    uint4 q[kTileVecs];
    uint32_t ok[kTileVecs], w = 0, n = 0;
    const bool some = load_tile(u, q, ok);
    if (plain) {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k) {
        float z[N];
        unpack16(q[k], z, T());
        if (some) {
#pragma unroll
          for (int i = 0; i < N; ++i) z[i] = ok[k] >> i & 1 ? z[i] : dead;
          n += __popc(ok[k]);
        }
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const uint2 b = raw_weights(z[i], z[i + 1], scale2, ymax2, zero2);
          w += b.x + b.y;
        }
      }
      w -= (uint32_t)(N * kTileVecs) * __float_as_uint(kUnit);
      if (!some) n = N * kTileVecs;
    } else {
#pragma unroll
      for (int k = 0; k < kTileVecs; ++k) {
        float z[N];
        unpack16(q[k], z, T());
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (some && !(ok[k] >> i & 1)) z[i] = kNegInf;
          w += token_weight(z[i], rs.scale, rs.ymax);
          n += z[i] > kNegInf ? 1u : 0u;
        }
      }
    }
    s.w += w;
    s.n += n;
    if constexpr (DECODE) {
      w = __reduce_add_sync(kFull, w);
      n = __reduce_add_sync(kFull, n);
      if (lane == 0) {
        if (ADJ && touch) {  // touched tokens are added by others
          atomicAdd(&tile_sums[tile].x, w);
          atomicAdd(&tile_sums[tile].y, n);
        } else {
          tile_sums[tile] = make_uint2(w, n);
        }
      }
    } else if (u + kTile <= u_target) {
      s.below_w += w;
      s.below_n += n;
    } else if (u <= u_target) {
      // the token's own tile: once per row
      for (int k = 0; k < kTileVecs; ++k) {
        const int u0 = u + k * kVecRow + lane * N;
        float z[N];
        fetch(u0, z, false);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t wi = token_weight(z[i], rs.scale, rs.ymax);
          const uint32_t ni = z[i] > kNegInf ? 1u : 0u;
          if (u0 + i < u_target) {
            s.below_w += wi;
            s.below_n += ni;
          }
          if (u0 + i == u_target && ni) peer_store(peer_address(&own_weight, 0), wi);
        }
      }
    }
  }, [&](int u, float z) {
    const uint32_t w = token_weight(z, rs.scale, rs.ymax);
    const uint32_t n = z > kNegInf ? 1u : 0u;
    s.w += w;
    s.n += n;
    if constexpr (DECODE) {
      atomicAdd(&tile_sums[(u - lo) / kTile].x, w);
      atomicAdd(&tile_sums[(u - lo) / kTile].y, n);
    } else {
      if (u < u_target) {
        s.below_w += w;
        s.below_n += n;
      }
      if (u == u_target && n) peer_store(peer_address(&own_weight, 0), w);
    }
  });
  const Sums sum = warp_total({s.w, s.n});
  Sums below = {0, 0};
  if constexpr (!DECODE) below = warp_total({s.below_w, s.below_n});
  if (lane < (DECODE ? (int)peers : 1)) {
    const uint32_t at = peer_address(&peer_sums[rank * warps + wid], lane);
    peer_store(at, sum.w);
    peer_store(at + 16, sum.n);
    if constexpr (!DECODE) {
      peer_store(at + 8, below.w);
      peer_store(at + 20, below.n);
    }
  }
  if (peers > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (!DECODE && (rank != 0 || wid != 0)) return;

  if (wid == 0) {
    // the row's sums; of the blocks before this one (below the token), and of
    // this one
    Sums all = {0, 0}, before = {0, 0}, mine = {0, 0};
    for (int i = lane; i < (int)peers * warps; i += 32) {
      const WarpSums p = peer_sums[i];
      all = all + Sums{p.w, p.n};
      if constexpr (DECODE) {
        if (i < (int)rank * warps) before = before + Sums{p.w, p.n};
        else if (i < (int)(rank + 1) * warps) mine = mine + Sums{p.w, p.n};
      } else {
        before = before + Sums{p.below_w, p.below_n};
      }
    }
    all = warp_total(all);
    before = warp_total(before);
    if constexpr (!DECODE) {
      if (lane != 0) return;
      if (own_weight == 0xffffffffu) return refuse(0, RANS_ERR_ZERO_FREQ, r, false);
      const uint32_t b = interval_start(before.w, before.n, all.w, all.n);
      starts[r] = b;
      freqs[r] = interval_start(before.w + own_weight, before.n + 1, all.w, all.n) - b;
      return;
    } else {
      // the block whose tokens hold the slot finds the tile that does, 32
      // tiles at a time
      const uint32_t slot = (uint32_t)x & (kTokTotal - 1);
      auto holds = [&](Sums at, Sums next) {
        return starts_by(at.w, at.n, all.w, all.n, slot) &&
               !starts_by(next.w, next.n, all.w, all.n, slot);
      };
      mine = warp_total(mine);
      int tile = -1;
      if (holds(before, before + mine)) {
        Sums base = before;
        const int tiles = (hi - lo + kTile - 1) / kTile;
        for (int t0 = 0; t0 < tiles && tile < 0; t0 += 32) {
          const uint2 own = t0 + lane < tiles ? tile_sums[t0 + lane] : make_uint2(0, 0);
          const Sums next = base + warp_scan({own.x, own.y}, lane);
          const Sums at = {next.w - own.x, next.n - own.y};
          const uint32_t hit = __ballot_sync(kFull, holds(at, next));
          if (hit) {
            const int l = __ffs(hit) - 1;
            tile = t0 + l;
            base.w = __shfl_sync(kFull, at.w, l);
            base.n = __shfl_sync(kFull, at.n, l);
          } else {
            base.w = __shfl_sync(kFull, next.w, 31);
            base.n = __shfl_sync(kFull, next.n, 31);
          }
        }
        if (lane == 0) {
          found_base = base;
          found_all = all;
        }
      }
      if (lane == 0) found_tile = tile;
    }
  }
  if constexpr (DECODE) {
    __syncthreads();
    const int tile = found_tile;
    if (tile < 0) return;
    const int u = lo + tile * kTile;
    // (tables start a whole number of spans after the block's first token)
    need_table(lo + (u - lo) / (dense ? kTouchSpan : kHashSpan) * (dense ? kTouchSpan : kHashSpan));
    if (wid != 0) return;
    const uint32_t slot = (uint32_t)x & (kTokTotal - 1);
    const Sums all = found_all;
    auto holds = [&](Sums at, Sums next) {
      return starts_by(at.w, at.n, all.w, all.n, slot) &&
             !starts_by(next.w, next.n, all.w, all.n, slot);
    };
    Sums base = found_base;
    for (int k = 0; k < kTileVecs; ++k) {
      const int u0 = u + k * kVecRow + lane * N;
      float z[N];
      fetch(u0, z, true);
      Sums own = {0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i)
        own = own + Sums{token_weight(z[i], rs.scale, rs.ymax), z[i] > kNegInf ? 1u : 0u};
      const Sums next = base + warp_scan(own, lane);
      Sums at = {next.w - own.w, next.n - own.n};
      if (holds(at, next)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (!(z[i] > kNegInf)) continue;
          const Sums after = {at.w + token_weight(z[i], rs.scale, rs.ymax), at.n + 1};
          if (holds(at, after)) {
            const uint32_t b = interval_start(at.w, at.n, all.w, all.n);
            take_token(cd, r, stream, x, taken, u0 + i - row.shift, b,
                       interval_start(after.w, after.n, all.w, all.n) - b, refill_ok,
                       refill_word, status);
          }
          at = after;
        }
      }
      base.w = __shfl_sync(kFull, next.w, 31);
      base.n = __shfl_sync(kFull, next.n, 31);
    }
  }
}

// --------------------------------------------------------------- streams --
// One warp per stream.  The states of a stream follow from one another, so the
// warp's lanes carry the same state; what does not depend on it is done 32
// tokens at a time, one per lane, a group ahead: loading the interval and
// turning the division by its freq into a product.  q = floor(x / f) for
// x < 2^63 is the high part of x times the ceiling of 2^(63 + l) / f,
// l = ceil(log2 f), shifted right by l (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994: exact since the factor
// exceeds 2^(63 + l) / f by less than 2^l / f).  What bounds the kernel is the
// chain of a step: compare, select, 64-bit product, shift, product, add.
// Measured: 64 streams of 64 tokens 14 us, and 4 us to compact them.
constexpr int kIntervalWarps = 4;
constexpr int kFusedStreams = 16;  // most streams of the one-block form

// What a step needs of its token.
struct Step {
  uint64_t inv;    // ceil(2^(63 + l) / freq)
  uint32_t freq;
  uint32_t start;  // | l << 24
};
static_assert(sizeof(Step) == 16, "one shared-memory load");

// floor(a 2^k / f) for f <= 2^24 and a quotient of at most 2^32, by a double
// quotient whose error is far below 1, and the remainder.
__device__ __forceinline__ uint64_t quotient(double a, uint64_t n, uint32_t f, double r,
                                             uint64_t &rem) {
  uint64_t q = (uint64_t)(a * r);
  int64_t left = (int64_t)(n - q * f);
  if (left < 0) {
    --q;
    left += f;
  } else if (left >= (int64_t)f) {
    ++q;
    left -= f;
  }
  rem = (uint64_t)left;
  return q;
}

__device__ __forceinline__ Step make_step(uint32_t start, uint32_t f) {
  const int l = f > 1 ? 32 - __clz(f - 1) : 0;
  const double r = 1.0 / (double)f;
  // 2^(63 + l) / f in two digits of 2^32
  const uint64_t top = 1ull << (31 + l);
  uint64_t r1, r2;
  const uint64_t q1 = quotient((double)top, top, f, r, r1);
  const uint64_t low = r1 << 32;
  const uint64_t q2 = quotient((double)low, low, f, r, r2);
  return {(q1 << 32) + q2 + (r2 ? 1u : 0u), f, start | (uint32_t)l << 24};
}

// Codes stream s into its scratch slot; returns its words (0: a bad extent).
__device__ __forceinline__ int64_t encode_stream(const uint32_t *__restrict__ starts,
                                                 const uint32_t *__restrict__ freqs,
                                                 const Geom &g, const StreamDesc &d, int64_t s,
                                                 uint32_t *end, Step *steps, int lane,
                                                 int32_t *status) {
  uint64_t x = kL;
  int64_t used = 0;
  auto load = [&](int64_t hi, uint32_t &st, uint32_t &f) {
    st = 0;
    f = 1;
    if (lane < hi) {
      st = starts[d.base + hi - 1 - lane];
      f = freqs[d.base + hi - 1 - lane];
    }
  };
  auto prepare = [&](uint32_t st, uint32_t f) {
    if (f == 0 || f > kTokTotal || st > kTokTotal - f) {
      report(status, f == 0 ? RANS_ERR_ZERO_FREQ : RANS_ERR_RANGE, s);
      st = 0;
      f = 1;
    }
    return make_step(st, f);
  };
  uint32_t st, f;
  load(d.n, st, f);
  Step mine = prepare(st, f);
  load(d.n - 32, st, f);
  for (int64_t hi = d.n; hi > 0; hi -= 32) {
    const int count = hi < 32 ? (int)hi : 32;
    __syncwarp();
    steps[lane] = mine;
    __syncwarp();
    uint32_t word = 0;
    int emitted = 0;
    auto take = [&](const Step &p) {
      // x >= 2^39 f, in the high words
      const bool emit = (uint32_t)(x >> 32) >= p.freq << 7;
      if (emit) {
        if (lane == emitted) word = (uint32_t)x;
        x >>= 32;
        ++emitted;
      }
      const uint64_t q = __umul64hi(x + x, p.inv) >> (p.start >> 24);
      x += (uint64_t)(p.start & (kTokTotal - 1)) + q * (uint64_t)(kTokTotal - p.freq);
    };
    if (count == 32) {
#pragma unroll 8
      for (int i = 0; i < 32; ++i) take(steps[i]);
    } else {
      for (int i = 0; i < count; ++i) take(steps[i]);
    }
    if (lane < emitted) end[-1 - used - lane] = word;
    used += emitted;
    mine = prepare(st, f);
    load(hi - 64, st, f);
  }
  if (lane == 0) {
    end[-1 - used] = (uint32_t)(x >> 32);
    end[-2 - used] = (uint32_t)x;
  }
  return used + 2;
}

// Whether a stream's extent lies within the scratch (slots are laid out from
// the first stream's start on).
__device__ __forceinline__ bool extent_ok(const Geom &g, const StreamDesc &d, int64_t s,
                                          int lane, int32_t *status) {
  const bool ok =
      d.ok && (g.kind != RANS_CHUNK_EXPLICIT || (g.starts[0] >= 0 && d.base >= g.starts[0]));
  if (!ok && lane == 0) report(status, RANS_ERR_ARG, s);
  return ok;
}

__global__ void __launch_bounds__(kIntervalWarps * 32)
    encode_intervals_kernel(const uint32_t *__restrict__ starts,
                            const uint32_t *__restrict__ freqs, Geom g, char *scratch,
                            uint64_t *lens, int32_t *status) {
  __shared__ Step steps[kIntervalWarps][32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t s = (int64_t)blockIdx.x * kIntervalWarps + wid;
  if (s >= g.S) return;
  const StreamDesc d = stream_desc(g, s);
  if (!extent_ok(g, d, s, lane, status)) return;
  uint32_t *end = reinterpret_cast<uint32_t *>(scratch + slot_end(g, d, s));
  const int64_t words =
      encode_stream(starts, freqs, g, d, s, end, steps[wid], lane, status);
  if (lane == 0) lens[s] = 4ull * (uint64_t)words;
}

// Few streams in one block: status, streams, offsets and compaction in one
// launch (two otherwise, and a memset): a text of 100 tokens, from logits to
// bytes, went from 37 to 26 us.  With more than kFusedStreams warps the chains
// would share a scheduler.
__global__ void __launch_bounds__(kFusedStreams * 32)
    encode_fused_kernel(const uint32_t *__restrict__ starts, const uint32_t *__restrict__ freqs,
                        Geom g, char *scratch, uint8_t *out, uint64_t capacity,
                        uint64_t *offsets, int32_t *status) {
  __shared__ Step steps[kFusedStreams][32];
  __shared__ uint64_t lens[kFusedStreams];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (threadIdx.x < (int)(sizeof(StatusWord) / 4)) status[threadIdx.x] = 0;
  __threadfence_block();
  __syncthreads();
  const StreamDesc d = stream_desc(g, wid);
  uint32_t *end = nullptr;
  int64_t words = 0;
  if (extent_ok(g, d, wid, lane, status)) {
    end = reinterpret_cast<uint32_t *>(scratch + slot_end(g, d, wid));
    words = encode_stream(starts, freqs, g, d, wid, end, steps[wid], lane, status);
  }
  if (lane == 0) lens[wid] = 4ull * (uint64_t)words;
  __syncthreads();
  uint64_t off = 0;
  for (int w = 0; w < wid; ++w) off += lens[w];
  const uint64_t to = off + 4ull * (uint64_t)words;
  if (lane == 0) {
    offsets[wid + 1] = to;
    if (wid == 0) offsets[0] = 0;
    if (wid == (int)g.S - 1 && to > capacity) report(status, RANS_ERR_CAPACITY, -1);
  }
  if (to > capacity) return;
  __syncwarp();  // the stream's words, written by the warp's lanes
  uint32_t *dst = reinterpret_cast<uint32_t *>(out + off);
  for (int64_t i = lane; i < words; i += 32) dst[i] = end[i - words];
}

__global__ void token_states_kernel(const uint8_t *in, uint64_t in_bytes,
                                    const uint64_t *offsets, int64_t S, uint64_t *states,
                                    int32_t *status) {
  const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= S) return;
  const uint64_t off = offsets[k], lim = offsets[k + 1];
  uint64_t x = 0;
  if (!(off & 3) && off <= lim && lim <= in_bytes && lim - off >= 8) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(in + off);
    x = (uint64_t)w[1] << 32 | w[0];
  }
  if (x < kL || x >> 63) {
    report(status, RANS_ERR_CORRUPT, k);
    x = 0;
  }
  states[2 * k] = x;
  states[2 * k + 1] = 2;
}

__global__ void token_finish_kernel(const uint64_t *offsets, int64_t S, const uint64_t *states,
                                    int32_t *status) {
  const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= S) return;
  if (states[2 * k] != kL || states[2 * k + 1] * 4 != offsets[k + 1] - offsets[k])
    report(status, RANS_ERR_CORRUPT, k);
}

// Blocks per row: one, while the rows alone fill the SMs; twice as many as
// long as all blocks would still run at once (two an SM) and each keeps a tile
// for eight warps.  (More, for finer shares: 256 rows of 131072 took 50 us with
// two blocks each and 53 with four, 43 with one.)
struct RowShape {
  int peers, threads, slice;
};
constexpr int kFewWarps = 8;

RowShape row_shape(int64_t rows, int tokens, int tile, int most, int sms) {
  const int tiles = (tokens + tile - 1) / tile;
  auto per = [&](int peers) { return (tiles + peers - 1) / peers; };
  int peers = 1;
  while (peers < most && rows * peers * 2 <= 2 * sms && per(peers * 2) >= kFewWarps)
    peers *= 2;
  const int warps = per(peers) < kRowWarps ? per(peers) : kRowWarps;
  return {peers, warps * 32, per(peers) * tile};
}

template <typename T, bool DECODE>
int launch_rows_t(const rans_logits &in, const rans_adjust &adj, const int32_t *tokens,
                  uint32_t *starts, uint32_t *freqs, const Coded &cd, int32_t *status,
                  cudaStream_t st) {
  const bool touch = adj.history != nullptr || adj.bias_ids != nullptr;
  auto kern = touch || adj.mask ? token_rows_kernel<T, DECODE, true>
                                : token_rows_kernel<T, DECODE, false>;
  const bool adjusted = touch || adj.mask;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RANS_ERR_CUDA;
  const int tile = 32 * VecOf<T>::N * row_vecs(adjusted);
  // rows that all start on 16 bytes have no empty places before them
  const bool aligned = reinterpret_cast<uintptr_t>(in.data) % 16 == 0 &&
                       (in.rows == 1 || in.row_stride % VecOf<T>::N == 0);
  if (ensure_cluster((const void *)kern) != cudaSuccess) return RANS_ERR_CUDA;
  // clusters of 16 need a processor group with 16 multiprocessors free of
  // defects; where a launch finds none, 8 are always to be had
  for (int most = kMaxCluster;; most = 8) {
    const RowShape shape = row_shape(in.rows, in.vocab + (aligned ? 0 : VecOf<T>::N - 1), tile,
                                     most, num_sms(dev));
    const uint32_t smem = (adjusted ? (uint32_t)sizeof(TouchTable) + kHashSpan / 8 : 0u) +
                          (DECODE ? (uint32_t)(shape.slice / tile * sizeof(uint2)) : 0u);
    if (smem && ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
    if (in.rows > 0x7fffffff / shape.peers) return RANS_ERR_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(in.rows * shape.peers));
    cfg.blockDim = dim3((unsigned)shape.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)shape.peers;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, in, adj, tokens, starts, freqs, cd, status, shape.slice,
                           (uint64_t)0x8000000080000000ull) == cudaSuccess)
      return RANS_OK;
    (void)cudaGetLastError();
    if (shape.peers <= 8) return RANS_ERR_CUDA;
  }
}

template <bool DECODE>
int launch_rows(const rans_logits &in, const rans_adjust &adj, const int32_t *tokens,
                uint32_t *starts, uint32_t *freqs, const Coded &cd, int32_t *status,
                cudaStream_t st) {
  switch (in.dtype) {
    case RANS_LOGITS_F32:
      return launch_rows_t<float, DECODE>(in, adj, tokens, starts, freqs, cd, status, st);
    case RANS_LOGITS_F16:
      return launch_rows_t<__half, DECODE>(in, adj, tokens, starts, freqs, cd, status, st);
    default:
      return launch_rows_t<__nv_bfloat16, DECODE>(in, adj, tokens, starts, freqs, cd, status, st);
  }
}

}  // namespace

int launch_token_intervals(const rans_logits &in, const rans_adjust &adj, const int32_t *tokens,
                           uint32_t *starts, uint32_t *freqs, int32_t *status, cudaStream_t st) {
  return launch_rows<false>(in, adj, tokens, starts, freqs, Coded(), status, st);
}

int launch_decode_tokens(const rans_logits &in, const rans_adjust &adj, const uint8_t *data,
                         uint64_t data_bytes, const uint64_t *offsets, int64_t S,
                         const int32_t *stream_ids, const uint64_t *states_in,
                         uint64_t *states_out, int32_t *tokens, int32_t *status,
                         cudaStream_t st) {
  const Coded cd = {data, data_bytes, offsets, S, stream_ids, states_in, states_out, tokens};
  return launch_rows<true>(in, adj, nullptr, nullptr, nullptr, cd, status, st);
}

int launch_encode_intervals(const uint32_t *starts, const uint32_t *freqs, const Geom &g,
                            char *ws, uint64_t header_bytes, uint64_t lens_bytes, uint8_t *out,
                            uint64_t capacity, uint64_t *offsets, cudaStream_t st) {
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  uint64_t *lens = reinterpret_cast<uint64_t *>(ws + header_bytes);
  char *scratch = ws + header_bytes + lens_bytes;
  if (g.S > 0 && g.S <= kFusedStreams) {
    encode_fused_kernel<<<1, (unsigned)g.S * 32, 0, st>>>(starts, freqs, g, scratch, out,
                                                          capacity, offsets, status);
    return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
  }
  if (cudaMemsetAsync(ws, 0, header_bytes + 8ull * (uint64_t)g.S, st) != cudaSuccess)
    return RANS_ERR_CUDA;
  if (g.S > 0) {
    const int64_t blocks = (g.S + kIntervalWarps - 1) / kIntervalWarps;
    if (blocks > 0x7fffffff) return RANS_ERR_ARG;
    encode_intervals_kernel<<<(unsigned)blocks, kIntervalWarps * 32, 0, st>>>(
        starts, freqs, g, scratch, lens, status);
    if (cudaGetLastError() != cudaSuccess) return RANS_ERR_CUDA;
  }
  return launch_compact(g, scratch, lens, out, capacity, offsets, status, st);
}

int launch_token_states(const uint8_t *in, uint64_t in_bytes, const uint64_t *offsets, int64_t S,
                        uint64_t *states, int32_t *status, cudaStream_t st) {
  if ((S + 127) / 128 > 0x7fffffff) return RANS_ERR_ARG;
  token_states_kernel<<<(unsigned)((S + 127) / 128), 128, 0, st>>>(in, in_bytes, offsets, S,
                                                                   states, status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

int launch_token_finish(const uint64_t *offsets, int64_t S, const uint64_t *states,
                        int32_t *status, cudaStream_t st) {
  if ((S + 127) / 128 > 0x7fffffff) return RANS_ERR_ARG;
  token_finish_kernel<<<(unsigned)((S + 127) / 128), 128, 0, st>>>(offsets, S, states, status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

}  // namespace rb
