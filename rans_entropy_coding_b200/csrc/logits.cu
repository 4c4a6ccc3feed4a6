// logits.cu -- rans_adjust_logits: penalties, biases, masks and temperature
// applied to rows of logits.
#include "logits_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kAdjThreads = 256;

// One block per kTouchSpan elements of a row.
template <typename T, typename O, bool TOUCH, bool MASK>
__global__ void __launch_bounds__(kAdjThreads)
    adjust_kernel(rans_logits in, rans_adjust adj, O *out, int64_t out_stride, int spans) {
  extern __shared__ __align__(16) unsigned char smem[];
  TouchTable &table = *reinterpret_cast<TouchTable *>(smem);
  constexpr int N = VecOf<T>::N;
  const int64_t r = blockIdx.x / spans;
  const int u_lo = (int)(blockIdx.x % spans) * kTouchSpan;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  __shared__ RowAdjust a;
  if (threadIdx.x == 0) a = row_adjust(adj, r, in.vocab);
  __syncthreads();
  const int u_hi = min(u_lo + kTouchSpan, row.end());
  bool touch = false;
  if constexpr (TOUCH) {
    touch = a.touches();
    if (touch) fill_touch(table, a, row.shift, in.vocab, u_lo, u_hi, threadIdx.x, kAdjThreads);
  }
  O *o = out + r * out_stride - row.shift;
  for (int u0 = u_lo + (int)threadIdx.x * N; u0 < u_hi; u0 += kAdjThreads * N) {
    float z[N];
    row.load(u0, z, 0.0f);
    if constexpr (TOUCH)
      if (touch) touch_vector<N>(z, table, a, u0 - u_lo);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = __fmul_rn(z[i], a.inv_temperature);
    if constexpr (MASK) mask_vector<N>(z, a, u0 - row.shift);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (u0 + i >= row.shift && u0 + i < row.end()) o[u0 + i] = float_logit<O>(z[i]);
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
  const int spans = (in.vocab + VecOf<T>::N - 1 + kTouchSpan - 1) / kTouchSpan;
  if (in.rows > 0x7fffffff / spans) return RANS_ERR_ARG;
  kern<<<(unsigned)(in.rows * spans), kAdjThreads, smem, st>>>(
      in, adj, static_cast<O *>(out), out_stride, spans);
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
