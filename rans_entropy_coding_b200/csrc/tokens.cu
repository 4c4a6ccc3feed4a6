// tokens.cu -- coding tokens under a model's logits: the intervals of given
// tokens (encoder side), one decoding step for a batch of streams, and the
// streams themselves.
//
// The weight of a token is an integer computed from its logit and the row's
// maximum by float32 operations that are each rounded on their own, so every
// kernel (and any other IEEE machine) gets the same one; all sums are of
// integers, so neither the split of a row over threads nor the order of
// additions can change an interval.
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

// max that keeps a NaN, so that one test per row finds it.
__device__ __forceinline__ float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
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
  if (zmax == kNegInf) {
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
constexpr int kTokThreads = 512;
constexpr int kTokWarps = kTokThreads / 32;
constexpr int kTokMaxSpans = RANS_MAX_VOCAB / kTouchSpan + 1;

struct Sums {
  uint64_t w;
  uint32_t n;
};

__device__ __forceinline__ Sums warp_sum(Sums s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.w += __shfl_xor_sync(kFull, s.w, o);
    s.n += __shfl_xor_sync(kFull, s.n, o);
  }
  return s;
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

// One block per row.  Pass 1 finds the row's maximum, pass 2 its sums; an
// encoding row also sums what lies below its token, a decoding row keeps the
// sums of every span and looks for its slot in the span that holds it.
template <typename T, bool DECODE>
__global__ void __launch_bounds__(kTokThreads)
    token_rows_kernel(rans_logits in, rans_adjust adj, const int32_t *tokens, uint32_t *starts,
                      uint32_t *freqs, Coded cd, int32_t *status) {
  extern __shared__ __align__(16) unsigned char smem[];
  TouchTable &table = *reinterpret_cast<TouchTable *>(smem);
  __shared__ float red_max[kTokWarps];
  __shared__ Sums red[kTokWarps], red2[kTokWarps];
  __shared__ Sums span_sum[kTokMaxSpans];
  __shared__ uint32_t own_weight;
  constexpr int N = VecOf<T>::N;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t r = blockIdx.x;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  const RowAdjust a = row_adjust(adj, r, in.vocab);
  const bool touch = a.touches();

  int target = -1;
  int64_t stream = r;
  uint64_t x = 0, taken = 0;
  if constexpr (DECODE) {
    if (cd.stream_ids) stream = cd.stream_ids[r];
    if (stream == -1) return;
    int bad = stream < 0 || stream >= cd.S;
    if (!bad && cd.stream_ids)
      for (int64_t i = tid; i < in.rows; i += kTokThreads)
        bad |= i != r && cd.stream_ids[i] == (int32_t)stream;
    bad = __syncthreads_or(bad);
    if (bad) {
      if (tid == 0) {
        report(status, RANS_ERR_INDEX, r);
        cd.tokens[r] = -1;
      }
      return;
    }
    x = cd.states_in[2 * stream];
    taken = cd.states_in[2 * stream + 1];
    __syncthreads();
    if (x < kL || x >> 63) {
      if (tid == 0) {
        report(status, RANS_ERR_CORRUPT, stream);
        cd.tokens[r] = -1;
        cd.states_out[2 * stream] = x;
        cd.states_out[2 * stream + 1] = taken;
      }
      return;
    }
  } else {
    target = tokens[r];
    if (target == -1) return;
    if (target < 0 || target >= in.vocab) {
      if (tid == 0) {
        report(status, RANS_ERR_INDEX, r);
        starts[r] = 0;
        freqs[r] = 0;
      }
      return;
    }
  }

  // the adjusted logits of the vector at u0
  auto fetch = [&](int u0, int u_lo, float (&z)[N]) {
    row.load(u0, z, kNegInf);
    if (touch) touch_vector<N>(z, table, a, u0 - u_lo);
    if (a.mask) mask_vector<N>(z, a, u0 - row.shift);
    if (!row.whole(u0)) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (u0 + i < row.shift || u0 + i >= row.end()) z[i] = kNegInf;
    }
  };

  float m = kNegInf;
  for (int u_lo = 0; u_lo < row.end(); u_lo += kTouchSpan) {
    if (touch) fill_touch(table, a, row.shift, in.vocab, u_lo, tid, kTokThreads);
    for (int u0 = u_lo + tid * N; u0 < min(u_lo + kTouchSpan, row.end()); u0 += kTokThreads * N) {
      float z[N];
      fetch(u0, u_lo, z);
#pragma unroll
      for (int i = 0; i < N; ++i) m = max_nan(m, z[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
  if (lane == 0) red_max[wid] = m;
  __syncthreads();
  m = red_max[0];
  for (int w = 1; w < kTokWarps; ++w) m = max_nan(m, red_max[w]);
  const RowScale rs = row_scale(m, a.inv_temperature);
  if (rs.error != RANS_OK) {
    if (tid == 0) {
      report(status, rs.error, r);
      if constexpr (DECODE) {
        cd.tokens[r] = -1;
        cd.states_out[2 * stream] = x;
        cd.states_out[2 * stream + 1] = taken;
      } else {
        starts[r] = 0;
        freqs[r] = 0;
      }
    }
    return;
  }

  const int u_target = row.shift + target;
  Sums all = {0, 0}, below = {0, 0};
  if (tid == 0) own_weight = 0xffffffffu;
  for (int u_lo = 0, span = 0; u_lo < row.end(); u_lo += kTouchSpan, ++span) {
    if (touch) fill_touch(table, a, row.shift, in.vocab, u_lo, tid, kTokThreads);
    else __syncthreads();
    Sums s = {0, 0};
    for (int u0 = u_lo + tid * N; u0 < min(u_lo + kTouchSpan, row.end()); u0 += kTokThreads * N) {
      float z[N];
      fetch(u0, u_lo, z);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t w = token_weight(z[i], rs.scale, rs.ymax);
        const uint32_t n = z[i] > kNegInf ? 1u : 0u;
        s.w += w;
        s.n += n;
        if constexpr (!DECODE) {
          if (u0 + i < u_target) {
            below.w += w;
            below.n += n;
          }
          if (u0 + i == u_target && n) own_weight = w;
        }
      }
    }
    all.w += s.w;
    all.n += s.n;
    if constexpr (DECODE) {
      s = warp_sum(s);
      if (lane == 0) red[wid] = s;
      __syncthreads();
      if (tid == 0) {
        Sums t = {0, 0};
        for (int w = 0; w < kTokWarps; ++w) {
          t.w += red[w].w;
          t.n += red[w].n;
        }
        span_sum[span] = t;
      }
    }
  }
  all = warp_sum(all);
  below = warp_sum(below);
  __syncthreads();
  if (lane == 0) {
    red[wid] = all;
    red2[wid] = below;
  }
  __syncthreads();
  all = red[0];
  below = red2[0];
  for (int w = 1; w < kTokWarps; ++w) {
    all.w += red[w].w;
    all.n += red[w].n;
    below.w += red2[w].w;
    below.n += red2[w].n;
  }

  if constexpr (!DECODE) {
    if (tid == 0) {
      if (own_weight == 0xffffffffu) {
        report(status, RANS_ERR_ZERO_FREQ, r);
        starts[r] = 0;
        freqs[r] = 0;
      } else {
        const uint32_t s = interval_start(below.w, below.n, all.w, all.n);
        starts[r] = s;
        freqs[r] = interval_start(below.w + own_weight, below.n + 1, all.w, all.n) - s;
      }
    }
  } else {
    const uint32_t slot = (uint32_t)x & (kTokTotal - 1);
    // the last span that starts at or before the slot
    Sums base = {0, 0};
    int span = 0;
    for (;; ++span) {
      if ((span + 1) * kTouchSpan >= row.end()) break;
      const Sums next = {base.w + span_sum[span].w, base.n + span_sum[span].n};
      if (!starts_by(next.w, next.n, all.w, all.n, slot)) break;
      base = next;
    }
    // warp 0 walks it, a warp's worth of vectors at a time.  The decoded token
    // is the last alive one that starts at or before the slot.
    const int u_lo = span * kTouchSpan;
    if (touch) fill_touch(table, a, row.shift, in.vocab, u_lo, tid, kTokThreads);
    if (wid != 0) return;
    bool done = false;
    for (int ub = u_lo; !done && ub < min(u_lo + kTouchSpan, row.end()); ub += 32 * N) {
      const int u0 = ub + lane * N;
      float z[N];
      if (u0 < row.end()) {
        fetch(u0, u_lo, z);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = kNegInf;
      }
      Sums mine = {0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        mine.w += token_weight(z[i], rs.scale, rs.ymax);
        mine.n += z[i] > kNegInf;
      }
      Sums incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t pw = __shfl_up_sync(kFull, incl.w, o);
        const uint32_t pn = __shfl_up_sync(kFull, incl.n, o);
        if (lane >= o) {
          incl.w += pw;
          incl.n += pn;
        }
      }
      Sums at = {base.w + incl.w - mine.w, base.n + incl.n - mine.n};
      const uint64_t end_w = __shfl_sync(kFull, base.w + incl.w, 31);
      const uint32_t end_n = __shfl_sync(kFull, base.n + incl.n, 31);
      // the token sits in this lane if an alive token of it contains the slot
      uint32_t s0 = 0, f0 = 0;
      int found = -1;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!(z[i] > kNegInf)) continue;
        const Sums next = {at.w + token_weight(z[i], rs.scale, rs.ymax), at.n + 1};
        if (starts_by(at.w, at.n, all.w, all.n, slot) &&
            !starts_by(next.w, next.n, all.w, all.n, slot)) {
          found = u0 + i - row.shift;
          s0 = interval_start(at.w, at.n, all.w, all.n);
          f0 = interval_start(next.w, next.n, all.w, all.n) - s0;
        }
        at = next;
      }
      if (found >= 0) {
        uint64_t y = (uint64_t)f0 * (x >> kTokPrec) + slot - s0;
        uint64_t used = taken;
        int token = found;
        if (y < kL) {
          const uint64_t off = cd.offsets[stream], lim = cd.offsets[stream + 1];
          const bool ok = !(off & 3) && off <= lim && lim <= cd.in_bytes &&
                          taken < (lim - off) / 4;
          if (ok) {
            y = y << 32 | reinterpret_cast<const uint32_t *>(cd.in)[off / 4 + taken];
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
      done = __any_sync(kFull, found >= 0);
      base.w = end_w;
      base.n = end_n;
    }
  }
}

// --------------------------------------------------------------- streams --
// One warp per stream.  The states of a stream follow from one another, so the
// warp's lanes carry the same state; what does not depend on it is done 32
// tokens at a time, one per lane: loading the interval and turning the
// division by its freq into a product.  q = floor(x / f) for x < 2^63 is the
// high part of x times the ceiling of 2^(63 + l) / f, l = ceil(log2 f), shifted
// right by l (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994: exact since the factor exceeds 2^(63 + l) / f by less
// than 2^l / f).
constexpr int kIntervalWarps = 4;

__global__ void __launch_bounds__(kIntervalWarps * 32)
    encode_intervals_kernel(const uint32_t *__restrict__ starts,
                            const uint32_t *__restrict__ freqs, Geom g, char *scratch,
                            uint64_t *lens, int32_t *status) {
  const int lane = threadIdx.x & 31;
  const int64_t s = (int64_t)blockIdx.x * kIntervalWarps + (threadIdx.x >> 5);
  if (s >= g.S) return;
  const StreamDesc d = stream_desc(g, s);
  // scratch slots are laid out from the first stream's start on
  if (!d.ok || (g.kind == RANS_CHUNK_EXPLICIT && (g.starts[0] < 0 || d.base < g.starts[0]))) {
    if (lane == 0) report(status, RANS_ERR_ARG, s);
    return;
  }
  uint32_t *end = reinterpret_cast<uint32_t *>(scratch + slot_end(g, d, s));
  uint64_t x = kL;
  int64_t used = 0;
  for (int64_t hi = d.n; hi > 0; hi -= 32) {
    const int count = hi < 32 ? (int)hi : 32;
    uint32_t st = 0, f = 1;
    if (lane < count) {
      st = starts[d.base + hi - 1 - lane];
      f = freqs[d.base + hi - 1 - lane];
      if (f == 0 || f > kTokTotal || st > kTokTotal - f) {
        report(status, f == 0 ? RANS_ERR_ZERO_FREQ : RANS_ERR_RANGE, s);
        st = 0;
        f = 1;
      }
    }
    const int l = f > 1 ? 32 - __clz(f - 1) : 0;
    const uint64_t top = 1ull << (31 + l);
    const uint64_t q1 = top / f, r1 = top - q1 * f;
    const uint64_t low = r1 << 32;
    const uint64_t q2 = low / f;
    const uint64_t inv = (q1 << 32) + q2 + (low != q2 * f ? 1 : 0);
    uint32_t word = 0;
    int emitted = 0;
    for (int i = 0; i < count; ++i) {
      const uint32_t fi = __shfl_sync(kFull, f, i);
      const uint32_t si = __shfl_sync(kFull, st, i);
      const int li = __shfl_sync(kFull, l, i);
      const uint64_t mi = __shfl_sync(kFull, inv, i);
      // x >= 2^39 f, in the high words
      const bool emit = (uint32_t)(x >> 32) >= fi << 7;
      if (emit) {
        if (lane == emitted) word = (uint32_t)x;
        x >>= 32;
        ++emitted;
      }
      const uint64_t q = __umul64hi(x + x, mi) >> li;
      x += (uint64_t)si + q * (uint64_t)(kTokTotal - fi);
    }
    if (lane < emitted) end[-1 - used - lane] = word;
    used += emitted;
  }
  if (lane == 0) {
    end[-1 - used] = (uint32_t)(x >> 32);
    end[-2 - used] = (uint32_t)x;
    lens[s] = 4ull * (uint64_t)(used + 2);
  }
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

template <typename T>
int launch_rows_t(const rans_logits &in, const rans_adjust &adj, const int32_t *tokens,
                  uint32_t *starts, uint32_t *freqs, const Coded *cd, int32_t *status,
                  cudaStream_t st) {
  auto kern = cd ? token_rows_kernel<T, true> : token_rows_kernel<T, false>;
  const bool touch = adj.history != nullptr || adj.bias_ids != nullptr;
  const uint32_t smem = touch ? (uint32_t)sizeof(TouchTable) : 0u;
  if (smem && ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  if (in.rows > 0x7fffffff) return RANS_ERR_ARG;
  kern<<<(unsigned)in.rows, kTokThreads, smem, st>>>(in, adj, tokens, starts, freqs,
                                                     cd ? *cd : Coded(), status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

int launch_rows(const rans_logits &in, const rans_adjust &adj, const int32_t *tokens,
                uint32_t *starts, uint32_t *freqs, const Coded *cd, int32_t *status,
                cudaStream_t st) {
  switch (in.dtype) {
    case RANS_LOGITS_F32:
      return launch_rows_t<float>(in, adj, tokens, starts, freqs, cd, status, st);
    case RANS_LOGITS_F16:
      return launch_rows_t<__half>(in, adj, tokens, starts, freqs, cd, status, st);
    default:
      return launch_rows_t<__nv_bfloat16>(in, adj, tokens, starts, freqs, cd, status, st);
  }
}

}  // namespace

int launch_token_intervals(const rans_logits &in, const rans_adjust &adj, const int32_t *tokens,
                           uint32_t *starts, uint32_t *freqs, int32_t *status, cudaStream_t st) {
  return launch_rows(in, adj, tokens, starts, freqs, nullptr, status, st);
}

int launch_decode_tokens(const rans_logits &in, const rans_adjust &adj, const uint8_t *data,
                         uint64_t data_bytes, const uint64_t *offsets, int64_t S,
                         const int32_t *stream_ids, const uint64_t *states_in,
                         uint64_t *states_out, int32_t *tokens, int32_t *status,
                         cudaStream_t st) {
  const Coded cd = {data, data_bytes, offsets, S, stream_ids, states_in, states_out, tokens};
  return launch_rows(in, adj, nullptr, nullptr, nullptr, &cd, status, st);
}

int launch_encode_intervals(const uint32_t *starts, const uint32_t *freqs, const Geom &g,
                            char *scratch, uint64_t *lens, int32_t *status, cudaStream_t st) {
  const int64_t blocks = (g.S + kIntervalWarps - 1) / kIntervalWarps;
  if (blocks > 0x7fffffff) return RANS_ERR_ARG;
  encode_intervals_kernel<<<(unsigned)blocks, kIntervalWarps * 32, 0, st>>>(
      starts, freqs, g, scratch, lens, status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
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
