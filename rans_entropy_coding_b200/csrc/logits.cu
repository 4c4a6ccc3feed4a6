// logits.cu -- rans_adjust_logits: penalties, biases, masks and temperature
// applied to rows of logits.
#include "logits_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

// A block takes a run of a row's tiles.  kAdjThreads threads stream them, four
// vectors of 16 bytes each; where a history or biases are given, kTableThreads
// more gather and adjust the touched logits meanwhile, whose values then go
// over what the stream left in their places.  (That wait for window, table and
// logits is a chain of memory latencies; before the stream, it cost as much as
// the stream itself.)  In place, the touched logits have to be read first, and
// all threads wait for that.
// Measured, 256 x 131072 bf16: 22 us with a temperature alone (6.1 TB/s; copying
// the rows takes 25 us), 31 us with a mask, 41 us with histories of 1024 to 2048
// tokens, 51 us with everything (2.75 TB/s): the tables, whose window every
// block of a row reads, are what is left.
constexpr int kAdjThreads = 512;
constexpr int kAdjVecs = 4;
constexpr int kTableThreads = 256;

template <typename T, typename O, bool TOUCH, bool MASK>
__global__ void __launch_bounds__(TOUCH ? kAdjThreads + kTableThreads : kAdjThreads, TOUCH ? 2 : 3)
    adjust_kernel(rans_logits in, rans_adjust adj, O *out, int64_t out_stride, int blocks,
                  int per_block) {
  extern __shared__ __align__(16) unsigned char smem[];
  TouchTable &table = *reinterpret_cast<TouchTable *>(smem);
  constexpr int N = VecOf<T>::N;
  constexpr int kTile = kAdjThreads * kAdjVecs * N;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t r = blockIdx.x / blocks;
  const Row<T> row(in.data, r, in.row_stride, in.vocab);
  const int lo = (int)(blockIdx.x % blocks) * per_block, hi = min(lo + per_block, row.end());
  if (lo >= hi) return;
  const uint32_t *mask = MASK ? adj.mask + r * adj.mask_stride : nullptr;
  const int words = (in.vocab + 31) >> 5;
  const float inv_temperature = adj.params ? adj.params[4 * r + 3] : adj.inv_temperature;
  O *o = out + r * out_stride - row.shift;  // element u goes to o[u]

  auto stream = [&](int from, int to) {
    constexpr int kWarpTile = 32 * kAdjVecs * N;
    for (int u = from + (tid >> 5) * kWarpTile; u < to; u += kTile) {
      const bool inside = u >= row.shift && u + kWarpTile <= row.end();
      uint4 q[kAdjVecs];
      uint32_t ok[kAdjVecs];
#pragma unroll
      for (int k = 0; k < kAdjVecs; ++k) {
        const int u0 = u + (32 * k + lane) * N;
        if (inside || row.whole(u0)) q[k] = *reinterpret_cast<const uint4 *>(row.at0 + u0);
      }
      if constexpr (MASK) {
#pragma unroll
        for (int k = 0; k < kAdjVecs; ++k)
          ok[k] = load_mask<N>(mask, words, u + 32 * k * N - row.shift, lane);
      }
#pragma unroll
      for (int k = 0; k < kAdjVecs; ++k) {
        const int u0 = u + (32 * k + lane) * N;
        float z[N];
        if (inside || row.whole(u0)) unpack16(q[k], z, T());
        else row.load(u0, z, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = __fmul_rn(z[i], inv_temperature);
        if constexpr (MASK) {
          const uint32_t bits = lane_mask<N>(ok[k], u + 32 * k * N - row.shift, lane);
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (!(bits >> i & 1)) z[i] = kNegInf;
        }
        if constexpr (sizeof(O) == sizeof(T)) {
          q[k] = pack16(z, O());
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (u0 + i >= row.shift && u0 + i < to) o[u0 + i] = float_logit<O>(z[i]);
        }
      }
      if constexpr (sizeof(O) == sizeof(T))
        store_tile<false>(o, u, q, inside, row.shift, to);
    }
  };
  if constexpr (!TOUCH) {
    stream(lo, hi);
  } else {
    __shared__ RowAdjust a;
    __shared__ bool table_dense;
    constexpr int kAll = kAdjThreads + kTableThreads;
    auto all = [] { __syncthreads(); };
    auto write_touched = [&] {
      each_touched(table, tid, kAll, [&](int u, float z) {
        o[u] = float_logit<O>(__fmul_rn(z, inv_temperature));
      });
    };
    bool dense = false;
    int u_lo = lo;
    if (static_cast<const void *>(out) != in.data) {
      if (tid < kAdjThreads) {
        stream(lo, hi);
      } else {
        auto among = [] { asm volatile("bar.sync 1, %0;" ::"n"(kTableThreads) : "memory"); };
        if (tid == kAdjThreads) a = row_adjust(adj, r, in.vocab);
        among();
        if (a.touches())
          fill_touch(table, a, row, lo, hi, dense, nullptr, tid - kAdjThreads, kTableThreads,
                     among);
        if (tid == kAdjThreads) table_dense = dense;
      }
      __syncthreads();
      if (!a.touches()) return;
      write_touched();
      dense = table_dense;
      // what the first table does not cover
      u_lo = lo + table.span;
      while (u_lo < hi) {
        u_lo += fill_touch(table, a, row, u_lo, hi, dense, nullptr, tid, kAll, all);
        write_touched();
      }
    } else {
      if (tid == 0) a = row_adjust(adj, r, in.vocab);
      __syncthreads();
      while (u_lo < hi) {
        const int from = u_lo;
        if (a.touches()) u_lo += fill_touch(table, a, row, from, hi, dense, nullptr, tid, kAll, all);
        else u_lo = hi;
        if (tid < kAdjThreads) stream(from, u_lo);
        __syncthreads();
        if (a.touches()) write_touched();
      }
    }
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
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RANS_ERR_CUDA;
  constexpr int kTile = kAdjThreads * kAdjVecs * VecOf<T>::N;
  const int tiles = (in.vocab + VecOf<T>::N - 1 + kTile - 1) / kTile;
  // tiles per block: one, until there are kAdjBlocks blocks for every SM (256
  // rows of 131072 with everything in use: 6 blocks an SM 51 us, 4 52 us, 2 81 us)
  constexpr int kAdjBlocks = 6;
  int64_t per = in.rows * tiles / ((int64_t)kAdjBlocks * num_sms(dev));
  per = per < 1 ? 1 : per > tiles ? tiles : per;
  const int blocks = (int)((tiles + per - 1) / per);
  if (in.rows > 0x7fffffff / blocks) return RANS_ERR_ARG;
  kern<<<(unsigned)(in.rows * blocks), touch ? kAdjThreads + kTableThreads : kAdjThreads, smem,
         st>>>(in, adj, static_cast<O *>(out), out_stride, blocks, (int)per * kTile);
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
