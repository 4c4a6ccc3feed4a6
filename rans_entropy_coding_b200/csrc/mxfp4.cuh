// mxfp4.cuh -- rows of microscaled 4-bit numbers: where their codes and scales
// lie (include/rans_b200.h, rans_mxfp4).
#pragma once

#include <cstdint>

#include "rans_b200.h"

namespace rb {

constexpr int kMxBlock = 32;       // elements that share a scale
constexpr int kMxGroup = 128;      // columns of a tile of scales (four bytes a row)
constexpr int kMxTileRows = 128;   // its rows
constexpr int kMxTileBytes = 512;

__host__ __device__ __forceinline__ int64_t mx_row_bytes(int64_t cols) {
  return (cols + kMxBlock - 1) / kMxBlock * (kMxBlock / 2);
}
__host__ __device__ __forceinline__ int mx_groups(int64_t cols) {
  return (int)((cols + kMxGroup - 1) / kMxGroup);
}
// Offset of the four scale bytes of row r in group g of `groups`.
__host__ __device__ __forceinline__ int64_t mx_scale_at(int64_t r, int g, int groups) {
  return ((r / kMxTileRows) * groups + g) * kMxTileBytes + 16 * (r % 32) + 4 * (r % 128 / 32);
}

}  // namespace rb
