// logits.cu -- rans_adjust_logits: penalties, biases, masks and temperature
// applied to rows of logits.
#include "logits_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

// A block takes kAdjTile elements of a row, all loaded before anything else.
constexpr int kAdjThreads = 256;
constexpr int kAdjVecs = 4;

template <typename T, typename O, bool TOUCH, bool MASK>
__global__ void __launch_bounds__(kAdjThreads)
    adjust_kernel(rans_logits in, rans_adjust adj, O *out, int64_t out_stride, int blocks) {
  extern __shared__ __align__(16) unsigned char smem[];
  TouchTable &table = *reinterpret_cast<TouchTable *>(smem);
  constexpr int N = VecOf<T>::N;
  constexpr int kTile = kAdjThreads * kAdjVecs * N;
  static_assert(kTile <= kTouchSpan, "one table per block");
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / blocks;
  const int u_lo = (int)(blockIdx.x % blocks) * kTile;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  const int u_hi = min(u_lo + kTile, row.end());
  uint4 q[kAdjVecs];
#pragma unroll
  for (int k = 0; k < kAdjVecs; ++k) {
    const int u0 = u_lo + (k * kAdjThreads + tid) * N;
    if (row.whole(u0)) q[k] = *reinterpret_cast<const uint4 *>(row.at0 + u0);
  }
  const uint32_t *mask = MASK ? adj.mask + r * adj.mask_stride : nullptr;
  const int words = (in.vocab + 31) >> 5;
  uint32_t ok[kAdjVecs];
  if constexpr (MASK) {
#pragma unroll
    for (int k = 0; k < kAdjVecs; ++k)
      ok[k] = mask_bits(mask, words, u_lo + (k * kAdjThreads + tid) * N - row.shift);
  }
  const float inv_temperature = adj.params ? adj.params[4 * r + 3] : adj.inv_temperature;
  bool touch = false;
  if constexpr (TOUCH) {
    __shared__ RowAdjust a;
    if (tid == 0) a = row_adjust(adj, r, in.vocab);
    __syncthreads();
    touch = a.touches();
    if (touch) fill_touch(table, a, row, u_lo, u_hi, tid, kAdjThreads);
  }
  O *o = out + r * out_stride - row.shift;  // element u goes to o[u]
  const bool aligned = (reinterpret_cast<uintptr_t>(o + u_lo) & 15) == 0 && sizeof(O) == sizeof(T);
#pragma unroll
  for (int k = 0; k < kAdjVecs; ++k) {
    const int u0 = u_lo + (k * kAdjThreads + tid) * N;
    if (u0 >= u_hi) break;
    float z[N];
    const bool whole = row.whole(u0);
    if (whole) unpack16(q[k], z, T());
    else row.load(u0, z, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      z[i] = __fmul_rn(z[i], inv_temperature);
      if (MASK && !(ok[k] >> i & 1)) z[i] = kNegInf;
    }
    if (whole && aligned) {
      if constexpr (sizeof(O) == sizeof(T))
        *reinterpret_cast<uint4 *>(o + u0) = pack16(z, O());
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (u0 + i >= row.shift && u0 + i < row.end()) o[u0 + i] = float_logit<O>(z[i]);
    }
  }
  if constexpr (TOUCH) {
    if (!touch) return;
    __syncthreads();  // the touched tokens' final values go over what stands there
    each_touched(table, tid, kAdjThreads, [&](int u, float z) {
      o[u] = float_logit<O>(__fmul_rn(z, inv_temperature));
    });
  }
}

template <typename T, typename O>
int launch_adjust_t(const rans_logits &in, const rans_adjust &adj, void *out, int64_t out_stride,
                    cudaStream_t st) {
  const bool touch = adj.history != nullptr || adj.bias_ids != nullptr;
  auto kern = touch ? (adj.mask ? adjust_kernel<T, O, true, true> : adjust_kernel<T, O, true, false>)
                    : (adj.mask ? adjust_kernel<T, O, false, true>
                                : adjust_kernel<T, O, false, false>);
  const uint32_t smem = touch ? (uint32_t)sizeof(TouchTable) : 0u;
  if (smem && ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  constexpr int kTile = kAdjThreads * kAdjVecs * VecOf<T>::N;
  const int blocks = (in.vocab + VecOf<T>::N - 1 + kTile - 1) / kTile;
  if (in.rows > 0x7fffffff / blocks) return RANS_ERR_ARG;
  kern<<<(unsigned)(in.rows * blocks), kAdjThreads, smem, st>>>(
      in, adj, static_cast<O *>(out), out_stride, blocks);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename T>
int launch_adjust_o(const rans_logits &in, const rans_adjust &adj, void *out, int out_dtype,
                    int64_t out_stride, cudaStream_t st) {
  switch (out_dtype) {
    case RANS_LOGITS_F32: return launch_adjust_t<T, float>(in, adj, out, out_stride, st);
    case RANS_LOGITS_F16: return launch_adjust_t<T, __half>(in, adj, out, out_stride, st);
    default: return launch_adjust_t<T, __nv_bfloat16>(in, adj, out, out_stride, st);
  }
}

}  // namespace

int launch_adjust(const rans_logits &in, const rans_adjust &adj, void *out, int out_dtype,
                  int64_t out_stride, cudaStream_t st) {
  switch (in.dtype) {
    case RANS_LOGITS_F32: return launch_adjust_o<float>(in, adj, out, out_dtype, out_stride, st);
    case RANS_LOGITS_F16: return launch_adjust_o<__half>(in, adj, out, out_dtype, out_stride, st);
    default: return launch_adjust_o<__nv_bfloat16>(in, adj, out, out_dtype, out_stride, st);
  }
}

}  // namespace rb
