// mxfp4.cu -- rows of floats to microscaled 4-bit numbers and back.
//
// A block of 32 elements shares a scale 2^(floor(log2 largest) - 2), so that
// the largest falls on [4, 8) and the elements on the eight magnitudes of a
// sign, two exponent bits and one of mantissa (up to 6, where larger ones
// saturate).  The exponent comes from the largest's bits; multiplying by the
// scale's inverse is exact (a power of two, and blocks' largest elements are
// never made subnormal by it), so an element is rounded once, by the
// hardware's conversion, to nearest with ties to even.
// Both directions are one pass over the rows and bound by memory.
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

// A warp takes kQuantVecs runs of 32 vectors, one after another along a row.
template <typename T>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_kernel(const T *x, int64_t rows, int64_t cols, int64_t stride, uint8_t *codes,
                    uint8_t *scales, int64_t units, int per_row) {
  constexpr int N = VecOf<T>::N;
  constexpr int kLanes = kMxBlock / N;  // lanes of a block
  constexpr int kRun = 32 * N;
  // (a product behind this launch may prepare itself meanwhile)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int64_t r = unit / per_row;
  const int64_t c0 = (unit - r * per_row) * (kRun * kQuantVecs);
  const T *row = x + r * stride, *end = row + cols;
  const int64_t row_bytes = mx_row_bytes(cols), padded = row_bytes * 2;
  const int groups = mx_groups(cols);
  uint4 q[kQuantVecs];
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    const int64_t c = c0 + k * kRun + lane * N;
    q[k] = c < cols ? load_joined(row, row + c, end) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    const int64_t c = c0 + k * kRun + lane * N;
    float z[N];
    unpack16(q[k], z, T());
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(z[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = scale_byte(top);
    const float inv = inverse_scale(byte);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = __fmul_rn(z[i], inv);
    const uint32_t w = codes8(z);
    if (c < padded) {
      uint8_t *at = codes + r * row_bytes + c / 2;
      if constexpr (N == 8) *reinterpret_cast<uint32_t *>(at) = w;
      else *reinterpret_cast<uint16_t *>(at) = (uint16_t)w;
    }
    // (bytes of a group's blocks past the row's end are 0)
    const int g = (int)(c / kMxGroup);
    if (lane % kLanes == 0 && g < groups)
      scales[mx_scale_at(r, g, groups) + c % kMxGroup / kMxBlock] = (uint8_t)byte;
  }
}

// Eight codes (or four, in the low half) as their magnitudes' floats: a code's
// exponent and mantissa bits become a float's, whose scale 2^126 undoes that the
// smallest magnitude is a subnormal.
__device__ __forceinline__ float code_value(uint32_t c) {
  const float a = __fmul_rn(__uint_as_float((c & 7u) << 22), 0x1p+126f);
  return __uint_as_float(__float_as_uint(a) | (c & 8u) << 28);
}

template <typename O>
__global__ void __launch_bounds__(32 * kQuantWarps)
    values_kernel(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, O *out,
                  int64_t stride, int64_t units, int per_row) {
  constexpr int N = VecOf<O>::N;
  constexpr int kRun = 32 * N;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int64_t r = unit / per_row;
  const int64_t c0 = (unit - r * per_row) * (kRun * kQuantVecs);
  const int64_t row_bytes = mx_row_bytes(cols), padded = row_bytes * 2;
  const int groups = mx_groups(cols);
  uint32_t w[kQuantVecs], byte[kQuantVecs];
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    const int64_t c = c0 + k * kRun + lane * N;
    w[k] = byte[k] = 0;
    if (c < padded) {
      const uint8_t *at = codes + r * row_bytes + c / 2;
      w[k] = N == 8 ? *reinterpret_cast<const uint32_t *>(at) : *reinterpret_cast<const uint16_t *>(at);
      byte[k] = scales[mx_scale_at(r, (int)(c / kMxGroup), groups) + c % kMxGroup / kMxBlock];
    }
  }
  uint4 p[kQuantVecs];
#pragma unroll
  for (int k = 0; k < kQuantVecs; ++k) {
    const float scale = byte[k] == 255u ? __int_as_float(0x7fffffff)
                        : byte[k] > 0  ? __uint_as_float(byte[k] << 23)
                                       : 0x1p-127f;
    float z[N];
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = __fmul_rn(code_value(w[k] >> (4 * i)), scale);
    p[k] = pack16(z, O());
  }
  const bool inside = c0 + kRun * kQuantVecs <= cols;
  // (columns fit an int: RANS_MAX_VOCAB of them at most)
  store_tile<false>(out + r * stride, (int)c0, p, inside, 0, (int)cols);
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
      static_cast<const T *>(x.data), x.rows, x.vocab, x.row_stride, q.codes, q.scales, u.units,
      u.per_row);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename O>
int values_t(const rans_mxfp4 &q, void *out, int64_t stride, cudaStream_t st) {
  const Units u = units_of(q.rows, q.cols, 32 * VecOf<O>::N);
  if (!u.ok) return RANS_ERR_ARG;
  values_kernel<O><<<u.blocks, 32 * kQuantWarps, 0, st>>>(
      q.codes, q.scales, q.rows, q.cols, static_cast<O *>(out), stride, u.units, u.per_row);
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
