// Descriptors and device helpers shared by the expert products
// (ciera_group.hip), the 4-bit operators (ciera_mx.hip) and their host side
// (ciera_ops.cpp).  Not part of the public ABI.
#pragma once
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace ciera {

constexpr uint32_t kMxBlock = 32;    // values behind one scale
constexpr uint32_t kMxColsPad = 128; // columns a 4-bit row is padded to
constexpr uint32_t kXcds = 8;        // compute dies; workgroup b starts on die b % 8

// Grouped product: out[i, n] = sum_k x[i, k] * W_g(i)[k, n].  Strides in elements.
struct GroupMmArgs {
  const void* x;
  const void* w;
  void* out;
  const int32_t* offsets;  // groups + 1 row offsets, or null: one group of all rows
  uint64_t ldx, ldw, ldo, gsw;
  int32_t rows, k, n, groups;
};

// Gradient of the weights: out_g[k, n] = sum over the group's rows of x[i, k] * dy[i, n].
struct GroupWgradArgs {
  const void* x;
  const void* dy;
  void* out;
  const int32_t* offsets;
  uint64_t ldx, ldy, ldo, gso;
  int32_t rows, k, n, groups;
};

// Product of 4-bit matrices: out[i, n] = sum_k a[i, k] * b_g(i)[n, k].
struct MxMmArgs {
  const uint8_t* a;
  const uint8_t* sa;
  const uint8_t* b;
  const uint8_t* sb;
  void* out;
  const int32_t* offsets;
  uint64_t ldo;
  int32_t rows, kp, n, groups;  // kp: padded columns
};

// x [groups][rows][cols] to codes and scales along axis 1 (rows of x are rows of the
// result) or axis 0 (columns of x are).
struct MxQuantArgs {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  uint64_t ldx, gsx;
  int32_t groups, rows, cols;  // of x
};

struct MxDequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  uint64_t ldo, gso;
  int32_t groups, rows, cols;
};

// Most row tiles of height bm that ascending offsets can make of `rows` rows.
inline uint64_t max_row_tiles(uint64_t rows, uint64_t groups, uint64_t bm) {
  if (groups == 1) return (rows + bm - 1) / bm;
  return rows / bm + (groups < rows ? groups : rows);
}
// The grid of one workgroup to a tile: as many on each die.
inline hipError_t tile_grid(uint64_t tiles, uint32_t threads, dim3* grid) {
  const uint64_t g = (tiles + kXcds - 1) / kXcds * kXcds;
  if (g * threads >> 32) return hipErrorInvalidConfiguration;
  *grid = dim3((uint32_t)g);
  return hipSuccess;
}
// Workgroups of the kernels that take one compute unit each.
constexpr uint32_t kUnits = 256;

// dtype: ciera_dtype_t of x; out_f32: the output is fp32 instead of x's type.
// flat: every operand row is 16-byte aligned (base, strides).
hipError_t launch_group_mm(int dtype, bool out_f32, bool transpose_w, bool flat, const GroupMmArgs& a, hipStream_t s);
hipError_t launch_group_wgrad(int dtype, bool out_f32, bool flat, const GroupWgradArgs& a, hipStream_t s);
hipError_t launch_mx_mm(int out_dtype, const MxMmArgs& a, hipStream_t s);
hipError_t launch_mx_quantize(int dtype, int axis, const MxQuantArgs& a, hipStream_t s);
hipError_t launch_mx_dequantize(int dtype, const MxDequantArgs& a, hipStream_t s);

}  // namespace ciera
