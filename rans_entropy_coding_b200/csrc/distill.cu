// distill.cu -- the coder's rate as a loss: distillation from a teacher's
// listed probabilities and tail, forward and backward.
//
// Write m for a maximum in logits, c = inv_temperature * log2(e).  The listed
// tokens are few: their terms are summed in double.  All others only enter
// through their own sum, kept against their own maximum, so that a student's
// small tail mass keeps its precision (1 - sum q would lose it):
//   R = sum over others of 2^(c (z - m_rest)),
//   Z = R 2^(c (m_rest - m)) + sum over listed of e^(inv_t (z_i - m)),
//   q_t = R 2^(c (m_rest - m)) / Z.
// The gradient of an unlisted token is then 2^(c (z - m_rest)) times one factor
// per row, inv_t (P q_t - p_t) / R, with no difference of close numbers per
// element.
#include <cmath>

#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kDisThreads = 512;
constexpr int kDisWarps = kDisThreads / 32;
constexpr double kLog2eD = 1.4426950408889634;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Per-row figures from the forward pass to the backward one (8 floats).
struct RowStats {
  float m_rest;    // largest logit of an unlisted token (0 if there is none)
  float rest;      // inv_t (P q_t - p_t) / R, the unlisted tokens' factor
  float m_all;     // largest logit of the row
  float inv_z;     // 1 / Z
  float mass;      // P
  float inv_p;     // 1 / sum p without a tail (0: no entry left), else 1
  float pad[2];
};
static_assert(sizeof(RowStats) == 32, "8 floats");

// Bits of the listed tokens by u; shared memory.  Reports an id outside the
// vocabulary or listed twice.  Every thread of the block calls it.
__device__ __forceinline__ void list_bits(uint32_t *bits, int words, const int32_t *ids,
                                          const float *lp, int K, int shift, int vocab,
                                          int64_t r, int32_t *status) {
  for (int i = threadIdx.x; i < words; i += kDisThreads) bits[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < K; i += kDisThreads) {
    const int v = ids[i];
    if (v == -1 || lp[i] == kNegInf) continue;
    if (v < 0 || v >= vocab) {
      if (status) report(status, RANS_ERR_INDEX, r);
      continue;
    }
    const int u = v + shift;
    const uint32_t old = atomicOr(&bits[u >> 5], 1u << (u & 31));
    if (status && (old >> (u & 31) & 1)) report(status, RANS_ERR_INDEX, r);
  }
  __syncthreads();
}

__device__ __forceinline__ bool entry(const int32_t *ids, const float *lp, int i, int vocab,
                                      int &v, float &l) {
  v = ids[i];
  l = lp[i];
  return v >= 0 && v < vocab && l != kNegInf;
}

// Sum over the block in a fixed order; every thread gets it.
template <typename X>
__device__ __forceinline__ X block_sum(X x, X *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  X t = red[0];
  for (int w = 1; w < kDisWarps; ++w) t += red[w];
  return t;
}

__device__ __forceinline__ float block_max(float x, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float t = red[0];
  for (int w = 1; w < kDisWarps; ++w) t = fmaxf(t, red[w]);
  return t;
}

// The row's loss and figures from the unlisted tokens' maximum and sum.
// Every thread calls it with the same m_rest and R.
template <typename T>
__device__ __forceinline__ void row_figures(const Row<T> &row, const int32_t *ids,
                                            const float *lp, int K, float inv_t, bool tail,
                                            float m_rest, double R, double *red, float *redf,
                                            float &loss, RowStats &st) {
  const T *z = row.at0 + row.shift;
  float m = m_rest;
  double sp = 0.0, count = 0.0;
  for (int i = threadIdx.x; i < K; i += kDisThreads) {
    int v;
    float l;
    if (!entry(ids, lp, i, row.vocab, v, l)) continue;
    m = fmaxf(m, logit_float(z[v]));
    sp += exp((double)l);
    count += 1.0;
  }
  m = block_max(m, redf);
  sp = block_sum(sp, red);
  count = block_sum(count, red);
  if (m == kNegInf) m = 0.0f;
  const double it = (double)inv_t;
  double top = 0.0;
  for (int i = threadIdx.x; i < K; i += kDisThreads) {
    int v;
    float l;
    if (entry(ids, lp, i, row.vocab, v, l))
      top += exp(((double)logit_float(z[v]) - (double)m) * it);
  }
  top = block_sum(top, red);
  const bool some = R > 0.0 || R != R;  // an unlisted token with a finite logit
  const double rest = some ? R * exp(((double)m_rest - (double)m) * it) : 0.0;
  const double Z = rest + top, lz = log(Z);
  const bool no_tail = !tail || count >= (double)row.vocab;
  const double norm = tail ? 1.0 : (sp > 0.0 ? 1.0 / sp : 0.0);
  const double pt = no_tail ? 0.0 : fmax(0.0, 1.0 - sp);
  const double mass = sp * norm + pt;
  double part = 0.0;
  const double lognorm = tail || !(sp > 0.0) ? 0.0 : -log(sp);
  for (int i = threadIdx.x; i < K; i += kDisThreads) {
    int v;
    float l;
    if (!entry(ids, lp, i, row.vocab, v, l)) continue;
    const double lpi = (double)l + lognorm;
    const double lq = ((double)logit_float(z[v]) - (double)m) * it - lz;
    const double p = exp(lpi);
    if (p > 0.0 || p != p) part += p * (lpi - lq);
  }
  part = block_sum(part, red);
  if (pt > 0.0) {
    const double lqt = some ? ((double)m_rest - (double)m) * it + log(R) - lz : -HUGE_VAL;
    part += pt * (log(pt) - lqt);
  }
  const bool ignored = !tail && !(sp > 0.0) && sp == sp;
  loss = ignored ? (Z == Z ? 0.0f : (float)Z) : (float)part;
  st.m_rest = some && m_rest > kNegInf ? m_rest : 0.0f;
  st.rest = some && !ignored ? (float)(it * (mass * (rest / Z) - pt) / R) : 0.0f;
  if (Z != Z) st.rest = (float)Z;
  st.m_all = m;
  st.inv_z = (float)(1.0 / Z);
  st.mass = (float)mass;
  st.inv_p = (float)norm;
  st.pad[0] = st.pad[1] = 0.0f;
}

template <typename T>
__device__ __forceinline__ void forward_row(const Row<T> &row, const uint32_t *bits,
                                            const int32_t *ids, const float *lp, int K,
                                            float inv_t, bool tail, double *red, float *redf,
                                            float &loss, RowStats &st) {
  constexpr int N = VecOf<T>::N;
  const float c = (float)((double)inv_t * kLog2eD);
  float m = kNegInf, s = 0.0f;
  for (int u0 = threadIdx.x * N; u0 < row.end(); u0 += kDisThreads * N) {
    float z[N];
    row.load(u0, z, kNegInf);
    const uint32_t hit = bits[u0 >> 5] >> (u0 & 31) & ((1u << N) - 1u);
    float vm = kNegInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (hit >> i & 1) z[i] = kNegInf;
      vm = fmaxf(vm, z[i]);
    }
    if (vm > m) {
      s *= exp2_fast((m - vm) * c);
      m = vm;
    }
    const float mz = m == kNegInf ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < N; ++i) s += exp2_fast((z[i] - mz) * c);
  }
  const float m_rest = block_max(m, redf);
  const double R =
      block_sum(m == kNegInf ? (double)s : (double)s * (double)exp2_fast((m - m_rest) * c), red);
  row_figures(row, ids, lp, K, inv_t, tail, m_rest, R, red, redf, loss, st);
}

// The gradient of a row, given its figures.
template <typename T>
__device__ __forceinline__ void backward_row(const Row<T> &row, const uint32_t *bits,
                                             const int32_t *ids, const float *lp, int K,
                                             float inv_t, const RowStats &st, float g, T *o,
                                             float *top_z) {
  constexpr int N = VecOf<T>::N;
  const float c = (float)((double)inv_t * kLog2eD);
  // grad may be the logits' own memory: the listed ones are read first
  for (int i = threadIdx.x; i < K; i += kDisThreads) {
    int v;
    float l;
    if (entry(ids, lp, i, row.vocab, v, l)) top_z[i] = logit_float(row.at0[row.shift + v]);
  }
  __syncthreads();
  const float factor = st.rest * g;
  for (int u0 = threadIdx.x * N; u0 < row.end(); u0 += kDisThreads * N) {
    float z[N];
    row.load(u0, z, kNegInf);
    const uint32_t hit = bits[u0 >> 5] >> (u0 & 31) & ((1u << N) - 1u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = u0 + i;
      if (u >= row.shift && u < row.end() && !(hit >> i & 1))
        o[u - row.shift] = float_logit<T>(exp2_fast((z[i] - st.m_rest) * c) * factor);
    }
  }
  for (int i = threadIdx.x; i < K; i += kDisThreads) {
    int v;
    float l;
    if (!entry(ids, lp, i, row.vocab, v, l)) continue;
    const float q = expf((top_z[i] - st.m_all) * inv_t) * st.inv_z;
    const float p = expf(l) * st.inv_p;
    o[v] = float_logit<T>((st.mass * q - p) * inv_t * g);
  }
}

template <typename T>
__global__ void __launch_bounds__(kDisThreads)
    distill_forward_kernel(rans_logits in, const int32_t *ids, const float *lp, int K,
                           float inv_t, int tail, float *losses, RowStats *stats,
                           int32_t *status) {
  extern __shared__ uint32_t bits[];
  __shared__ double red[kDisWarps];
  __shared__ float redf[kDisWarps];
  const int64_t r = blockIdx.x;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  ids += r * K;
  lp += r * K;
  const int words = (in.vocab + VecOf<T>::N + 31) / 32;
  list_bits(bits, words, ids, lp, K, row.shift, in.vocab, r, status);
  float loss;
  RowStats st;
  forward_row(row, bits, ids, lp, K, inv_t, tail != 0, red, redf, loss, st);
  if (threadIdx.x == 0) {
    losses[r] = loss;
    stats[r] = st;
  }
}

template <typename T>
__global__ void __launch_bounds__(kDisThreads)
    distill_backward_kernel(rans_logits in, const int32_t *ids, const float *lp, int K,
                            float inv_t, const RowStats *stats, const float *grads, T *grad,
                            int64_t grad_stride) {
  extern __shared__ uint32_t bits[];
  __shared__ float top_z[RANS_MAX_TOP];
  const int64_t r = blockIdx.x;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  ids += r * K;
  lp += r * K;
  const int words = (in.vocab + VecOf<T>::N + 31) / 32;
  list_bits(bits, words, ids, lp, K, row.shift, in.vocab, r, nullptr);
  backward_row(row, bits, ids, lp, K, inv_t, stats[r], grads[r], grad + r * grad_stride, top_z);
}

// Both in one launch: the row is read again for the gradient (from L2).
template <typename T>
__global__ void __launch_bounds__(kDisThreads)
    distill_both_kernel(rans_logits in, const int32_t *ids, const float *lp, int K, float inv_t,
                        int tail, const float *grads, float *losses, T *grad,
                        int64_t grad_stride, int32_t *status) {
  extern __shared__ uint32_t bits[];
  __shared__ double red[kDisWarps];
  __shared__ float redf[kDisWarps];
  __shared__ float top_z[RANS_MAX_TOP];
  const int64_t r = blockIdx.x;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  ids += r * K;
  lp += r * K;
  const int words = (in.vocab + VecOf<T>::N + 31) / 32;
  list_bits(bits, words, ids, lp, K, row.shift, in.vocab, r, status);
  float loss;
  RowStats st;
  forward_row(row, bits, ids, lp, K, inv_t, tail != 0, red, redf, loss, st);
  if (threadIdx.x == 0) losses[r] = loss;
  backward_row(row, bits, ids, lp, K, inv_t, st, grads[r], grad + r * grad_stride, top_z);
}

template <typename T>
uint32_t bits_bytes(int vocab) {
  return 4u * (uint32_t)((vocab + VecOf<T>::N + 31) / 32);
}

template <typename T>
int forward_t(const rans_logits &in, const int32_t *ids, const float *lp, int K, float inv_t,
              int tail, float *losses, float *stats, int32_t *status, cudaStream_t st) {
  auto kern = distill_forward_kernel<T>;
  const uint32_t smem = bits_bytes<T>(in.vocab);
  if (ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  kern<<<(unsigned)in.rows, kDisThreads, smem, st>>>(in, ids, lp, K, inv_t, tail, losses,
                                                     reinterpret_cast<RowStats *>(stats), status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename T>
int backward_t(const rans_logits &in, const int32_t *ids, const float *lp, int K, float inv_t,
               const float *stats, const float *grads, void *grad, int64_t stride,
               cudaStream_t st) {
  auto kern = distill_backward_kernel<T>;
  const uint32_t smem = bits_bytes<T>(in.vocab);
  if (ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  kern<<<(unsigned)in.rows, kDisThreads, smem, st>>>(
      in, ids, lp, K, inv_t, reinterpret_cast<const RowStats *>(stats), grads,
      static_cast<T *>(grad), stride);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename T>
int both_t(const rans_logits &in, const int32_t *ids, const float *lp, int K, float inv_t,
           int tail, const float *grads, float *losses, void *grad, int64_t stride,
           int32_t *status, cudaStream_t st) {
  auto kern = distill_both_kernel<T>;
  const uint32_t smem = bits_bytes<T>(in.vocab);
  if (ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  kern<<<(unsigned)in.rows, kDisThreads, smem, st>>>(in, ids, lp, K, inv_t, tail, grads, losses,
                                                     static_cast<T *>(grad), stride, status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

}  // namespace

int launch_distill_forward(const rans_logits &in, const int32_t *ids, const float *lp, int K,
                           float inv_t, int tail, float *losses, float *stats, int32_t *status,
                           cudaStream_t st) {
  if (in.rows > 0x7fffffff) return RANS_ERR_ARG;
  switch (in.dtype) {
    case RANS_LOGITS_F32:
      return forward_t<float>(in, ids, lp, K, inv_t, tail, losses, stats, status, st);
    case RANS_LOGITS_F16:
      return forward_t<__half>(in, ids, lp, K, inv_t, tail, losses, stats, status, st);
    default:
      return forward_t<__nv_bfloat16>(in, ids, lp, K, inv_t, tail, losses, stats, status, st);
  }
}

int launch_distill_backward(const rans_logits &in, const int32_t *ids, const float *lp, int K,
                            float inv_t, const float *stats, const float *grads, void *grad,
                            int64_t stride, cudaStream_t st) {
  if (in.rows > 0x7fffffff) return RANS_ERR_ARG;
  switch (in.dtype) {
    case RANS_LOGITS_F32:
      return backward_t<float>(in, ids, lp, K, inv_t, stats, grads, grad, stride, st);
    case RANS_LOGITS_F16:
      return backward_t<__half>(in, ids, lp, K, inv_t, stats, grads, grad, stride, st);
    default:
      return backward_t<__nv_bfloat16>(in, ids, lp, K, inv_t, stats, grads, grad, stride, st);
  }
}

int launch_distill(const rans_logits &in, const int32_t *ids, const float *lp, int K,
                   float inv_t, int tail, const float *grads, float *losses, void *grad,
                   int64_t stride, int32_t *status, cudaStream_t st) {
  if (in.rows > 0x7fffffff) return RANS_ERR_ARG;
  switch (in.dtype) {
    case RANS_LOGITS_F32:
      return both_t<float>(in, ids, lp, K, inv_t, tail, grads, losses, grad, stride, status, st);
    case RANS_LOGITS_F16:
      return both_t<__half>(in, ids, lp, K, inv_t, tail, grads, losses, grad, stride, status, st);
    default:
      return both_t<__nv_bfloat16>(in, ids, lp, K, inv_t, tail, grads, losses, grad, stride,
                                   status, st);
  }
}

}  // namespace rb
