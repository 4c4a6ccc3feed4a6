// mxfp4.cu -- rows of floats to microscaled 4-bit numbers and back.
//
// A block of 32 elements shares a scale 2^(floor(log2 largest) - 2), so that
// the largest falls on [4, 8) and the elements on the eight magnitudes of a
// sign, two exponent bits and one of mantissa (up to 6, where larger ones
// saturate).  The exponent comes from the largest's bits; multiplying by the
// scale's inverse is exact (a power of two, and blocks' largest elements are
// never made subnormal by it), so an element is rounded once, by the
// hardware's conversion, to nearest with ties to even.
// Both directions are one pass over the rows.  Measured, 131072 x 4096 bf16: to codes
// 244 us (5.6 TB/s), back 225 us (6.05 TB/s; copying runs at 6.55).
#include "logits_common.cuh"
#include "mxfp4.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kQuantWarps = 8;
constexpr int kQuantVecs = 4;  // vectors of 16 bytes in flight per lane

// Eight codes, element 0 in the low bits.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8]) {
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(c)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return c;
}
__device__ __forceinline__ uint32_t codes8(const float (&x)[4]) {
  const float y[8] = {x[0], x[1], x[2], x[3], 0.0f, 0.0f, 0.0f, 0.0f};
  return codes8(y);
}

// The scale byte of a block from the bits of its largest magnitude: the
// exponent less 2, not below 0; 255 (no number) where an element is infinite or
// no number.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255 ? 255u : e > 2 ? e - 2 : 0u;
}
// 2^(127 - byte): bytes are at most 252 but for 255, whose codes mean nothing.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float((byte > 252 ? 1u : 254u - byte) << 23);
}

// The bits of a float32 at least as large as the magnitudes of a vector's elements and
// with the largest one's exponent; an infinity or NaN where there is one.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const uint4 &q) {
  if constexpr (sizeof(T) == 2) {
    constexpr uint32_t kMagnitude = 0x7fff7fffu;
    const uint32_t m = pair_max(pair_max(q.x & kMagnitude, q.y & kMagnitude, T()),
                                pair_max(q.z & kMagnitude, q.w & kMagnitude, T()), T());
    float z[8];
    unpack16(make_uint4(m, 0, 0, 0), z, T());
    return max(__float_as_uint(z[0]), __float_as_uint(z[1]));
  } else {
    constexpr uint32_t kMagnitude = 0x7fffffffu;
    return max(max(q.x & kMagnitude, q.y & kMagnitude), max(q.z & kMagnitude, q.w & kMagnitude));
  }
}

// A warp takes kQuantVecs runs of 32 vectors, one after another along a row.
// Bound by the ALUs (77% busy: unpacking, maxima and conversions, 12 instructions an
// element) a little more than by memory.  With maxima of single elements and
// every run checked for the row's end it took 369 us.
template <typename T>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_kernel(const T *x, int64_t cols, int64_t stride, uint8_t *codes, uint8_t *scales,
                    int64_t units, int per_row) {
  constexpr int N = VecOf<T>::N;
  constexpr int kLanes = kMxBlock / N;  // lanes of a block
  constexpr int kRun = 32 * N;
  constexpr int kRunGroups = kRun / kMxGroup;
  // (a product behind this launch may prepare itself meanwhile)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int64_t r = unit / per_row;
  const int c0 = (int)(unit - r * per_row) * (kRun * kQuantVecs), c = c0 + lane * N;
  const T *row = x + r * stride;
  const int64_t row_bytes = mx_row_bytes(cols);
  const int groups = mx_groups(cols);
  uint8_t *code_at = codes + r * row_bytes + c / 2;
  uint8_t *scale_at = scales + mx_scale_at(r, c / kMxGroup, groups) + c % kMxGroup / kMxBlock;
  const bool whole = c0 + kRun * kQuantVecs <= cols;
  uint4 q[kQuantVecs];
  if (whole && reinterpret_cast<uintptr_t>(row) % 16 == 0) {
#pragma unroll
    for (int k = 0; k < kQuantVecs; ++k)
      q[k] = __ldcs(reinterpret_cast<const uint4 *>(row + c + k * kRun));
  } else {
#pragma unroll
    for (int k = 0; k < kQuantVecs; ++k)
      q[k] = c + k * kRun < cols ? load_joined(row, row + c + k * kRun, row + cols)
                                 : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    uint32_t top = top_bits<T>(q[k]);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = scale_byte(top);
    const float inv = inverse_scale(byte);
    float z[N];
    unpack16(q[k], z, T());
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = __fmul_rn(z[i], inv);
    const uint32_t w = codes8(z);
    if (whole || c + k * kRun < 2 * row_bytes) {
      if constexpr (N == 8) *reinterpret_cast<uint32_t *>(code_at + k * kRun / 2) = w;
      else *reinterpret_cast<uint16_t *>(code_at + k * kRun / 2) = (uint16_t)w;
    }
    // (bytes of a group's blocks past the row's end are 0)
    if (lane % kLanes == 0 && (whole || (c + k * kRun) / kMxGroup < groups))
      scale_at[k * kRunGroups * kMxTileBytes] = (uint8_t)byte;
  }
}

// The numbers of N codes.  (Each width unpacks a register of its own size: four bytes
// unpacked from a zero-extended half gave zeros.)
__device__ __forceinline__ void code_values(uint32_t w, float (&z)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
  unpack16(make_uint4(h[0], h[1], h[2], h[3]), z, __half());
}
__device__ __forceinline__ void code_values(uint32_t w, float (&z)[4]) {
  uint32_t h[2];
  asm("{\n\t.reg .b8 a, b;\n\tmov.b16 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "h"((uint16_t)w));
  float y[8];
  unpack16(make_uint4(h[0], h[1], 0, 0), y, __half());
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = y[i];
}

template <typename O>
__global__ void __launch_bounds__(32 * kQuantWarps)
    values_kernel(const uint8_t *codes, const uint8_t *scales, int64_t cols, O *out,
                  int64_t stride, int64_t units, int per_row) {
  constexpr int N = VecOf<O>::N;
  constexpr int kRun = 32 * N;
  constexpr int kRunGroups = kRun / kMxGroup;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int64_t r = unit / per_row;
  const int c0 = (int)(unit - r * per_row) * (kRun * kQuantVecs), c = c0 + lane * N;
  const int64_t row_bytes = mx_row_bytes(cols);
  const int groups = mx_groups(cols);
  const uint8_t *code_at = codes + r * row_bytes + c / 2;
  const uint8_t *scale_at = scales + mx_scale_at(r, c / kMxGroup, groups) + c % kMxGroup / kMxBlock;
  const bool whole = c0 + kRun * kQuantVecs <= cols;
  uint32_t w[kQuantVecs], byte[kQuantVecs];
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    w[k] = byte[k] = 0;
    if (whole || c + k * kRun < 2 * row_bytes) {
      if constexpr (N == 8) w[k] = *reinterpret_cast<const uint32_t *>(code_at + k * kRun / 2);
      else w[k] = *reinterpret_cast<const uint16_t *>(code_at + k * kRun / 2);
      byte[k] = scale_at[k * kRunGroups * kMxTileBytes];
    }
  }
  uint4 p[kQuantVecs];
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    const float scale = byte[k] == 255u ? __int_as_float(0x7fffffff)
                        : byte[k] > 0  ? __uint_as_float(byte[k] << 23)
                                       : 0x1p-127f;
    float z[N];
    code_values(w[k], z);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = __fmul_rn(z[i], scale);
    p[k] = pack16(z, O());
  }
  // (columns fit an int: RANS_MAX_VOCAB of them at most)
  store_tile<false>(out + r * stride, c0, p, whole, 0, (int)cols);
}

struct Units {
  int64_t units;
  int per_row;
  unsigned blocks;
  bool ok;
};
Units units_of(int64_t rows, int64_t cols, int run) {
  const int per_row = (int)((cols + run * kQuantVecs - 1) / (run * kQuantVecs));
  const int64_t units = rows * per_row, blocks = (units + kQuantWarps - 1) / kQuantWarps;
  return {units, per_row, (unsigned)blocks, blocks <= 0x7fffffff};
}

template <typename T>
int quantize_t(const rans_logits &x, const rans_mxfp4 &q, cudaStream_t st) {
  const Units u = units_of(x.rows, x.vocab, 32 * VecOf<T>::N);
  if (!u.ok) return RANS_ERR_ARG;
  quantize_kernel<T><<<u.blocks, 32 * kQuantWarps, 0, st>>>(
      static_cast<const T *>(x.data), x.vocab, x.row_stride, q.codes, q.scales, u.units, u.per_row);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename O>
int values_t(const rans_mxfp4 &q, void *out, int64_t stride, cudaStream_t st) {
  const Units u = units_of(q.rows, q.cols, 32 * VecOf<O>::N);
  if (!u.ok) return RANS_ERR_ARG;
  values_kernel<O><<<u.blocks, 32 * kQuantWarps, 0, st>>>(
      q.codes, q.scales, q.cols, static_cast<O *>(out), stride, u.units, u.per_row);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

}  // namespace

int launch_mxfp4_quantize(const rans_logits &x, const rans_mxfp4 &q, cudaStream_t st) {
  switch (x.dtype) {
    case RANS_LOGITS_F32: return quantize_t<float>(x, q, st);
    case RANS_LOGITS_F16: return quantize_t<__half>(x, q, st);
    default: return quantize_t<__nv_bfloat16>(x, q, st);
  }
}

int launch_mxfp4_values(const rans_mxfp4 &q, void *out, int dtype, int64_t stride,
                        cudaStream_t st) {
  switch (dtype) {
    case RANS_LOGITS_F32: return values_t<float>(q, out, stride, st);
    case RANS_LOGITS_F16: return values_t<__half>(q, out, stride, st);
    default: return values_t<__nv_bfloat16>(q, out, stride, st);
  }
}

}  // namespace rb
