// How the 4-bit operators pass over the rows of a matrix: loads of 8 values at any
// element, which lane takes what, grids.
#pragma once
#include "ciera_tiles.h"

namespace ciera {
namespace {

// 8 consecutive values as words, those from `left` on as zeros.
// (A branch to each of the last ones: 400000 rows of 31 values, bf16, 32.6 us for 24.2,
// 40000 of 1447 29.9 for 25.8.)
template <typename I>
__device__ __forceinline__ void load8(const typename I::T* p, int left, uint32_t* w) {
  constexpr int N = 8 / I::kPer;
  if (left >= 8) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const i32x4 v = load16(reinterpret_cast<const char*>(p) + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; j++) w[i + j] = v[j];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; i++) w[i] = 0;
  if (left <= 0) return;
  // all at once, the last one again in place of those behind it
  typename I::T v[8];
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = p[min(j, left - 1)];
#pragma unroll
  for (int j = 0; j < 8; j++) w[j / I::kPer] |= (j < left ? (uint32_t)v[j] : 0) << (I::kPer == 2 ? 16 * (j & 1) : 0);
}

// How a wave passes over rows in chunks of 8 values (16 bytes of a two-byte type, 4 of
// codes): a segment is 64 chunks of one row, or of 2 or 4 rows where these are that
// short; each wave takes kRun consecutive segments, so that as many loads are under way.
constexpr int kRun = 4;
struct RowPass {
  uint32_t width;   // lanes of a segment on one row, log2: 16, 32 or 64
  uint32_t chunks;  // of a row
  uint32_t segs;    // segments of a row (or of 64 / width rows)
  uint32_t narrow;  // segments and rows are 32-bit counts
  uint64_t lines, total;

  RowPass(uint64_t groups, uint64_t rows, uint64_t cols) {
    chunks = (uint32_t)((cols + kMxColsPad - 1) / kMxColsPad * (kMxColsPad / 8));
    width = chunks <= 16 ? 4 : chunks <= 32 ? 5 : 6;
    segs = (chunks + (1u << width) - 1) >> width;
    lines = groups * rows;
    const uint64_t at_once = 64 >> width;
    total = (lines + at_once - 1) / at_once * segs;
    narrow = total < 0xffffffffu - 4096 && lines < 0xffffffffu;
  }
  __device__ __forceinline__ uint64_t quotient(uint64_t n, uint32_t d) const {
    return narrow ? (uint32_t)n / d : n / d;
  }
  // this lane's row and chunk in segment s; false: none
  __device__ __forceinline__ bool locate(uint64_t s, uint64_t* line, uint32_t* chunk) const {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t l = segs == 1 ? s : quotient(s, segs);
    *chunk = ((uint32_t)(s - l * segs) << width) + (lane & ((1u << width) - 1));
    *line = (l << (6 - width)) + (lane >> width);
    return s < total && *line < lines && *chunk < chunks;
  }
};
__device__ __forceinline__ uint64_t first_segment() {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  return ((uint64_t)blockIdx.x * 4 + wave) * kRun;
}

// Workgroups of a pass; beyond the limit each takes several parts in turn.
uint32_t pass_grid(uint64_t parts, uint64_t limit) { return (uint32_t)(parts < limit ? parts : limit); }
uint32_t row_grid(const RowPass& p) { return pass_grid((p.total + 4 * kRun - 1) / (4 * kRun), 1 << 20); }

}  // namespace
}  // namespace ciera
