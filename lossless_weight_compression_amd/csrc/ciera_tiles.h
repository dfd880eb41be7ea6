// Device helpers of the matrix products: group search, LDS tile layout,
// fragment reads, matrix instructions, stores.
#pragma once
#include "ciera_ops_internal.h"

namespace ciera {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef __bf16 T;
  typedef bf16x8 V;
};
struct Fp16 {
  typedef _Float16 T;
  typedef f16x8 V;
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 16 bytes at any 2-byte aligned address (the hardware splits what crosses a line).
struct __attribute__((packed, aligned(2))) Bytes16 {
  i32x4 v;
};
__device__ __forceinline__ i32x4 load16(const void* p) { return reinterpret_cast<const Bytes16*>(p)->v; }

// The rows of one group as the kernel sees them: offsets out of order or out of
// range are clamped, so that no access leaves the operands.
__device__ __forceinline__ void group_range(const int32_t* off, int g, int rows, int* begin, int* count) {
  if (!off) {
    *begin = 0;
    *count = rows;
    return;
  }
  const int a = min(max(off[g], 0), rows), b = min(max(off[g + 1], 0), rows);
  *begin = a;
  *count = max(b - a, 0);
}

__device__ __forceinline__ int wave_inclusive_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Where workgroup `bid` of a product grouped by expert works: tile m of group g
// (rows [begin + m * bm, begin + count)) and column tile n.  The row tiles of all
// groups are numbered in order; each wave adds them up by itself, 64 groups at a
// time.  Workgroups are dealt to the dies in turn, so each die gets one
// contiguous run of the tiles: its L2 then holds few groups' weights at a time.
// The grid covers the largest possible number of tiles; false: nothing to do.
struct GroupTile {
  int g, m, n, begin, count;
};
__device__ __forceinline__ bool find_group_tile(const int32_t* off, int groups, int rows, int bm, int ntiles,
                                                uint32_t bid, GroupTile* t) {
  const int lane = threadIdx.x & 63;
  uint32_t total = 0;
  int begin = 0, count = 0, incl = 0;
  for (int c = 0; c < groups; c += 64) {
    begin = count = 0;
    if (c + lane < groups) group_range(off, c + lane, rows, &begin, &count);
    incl = wave_inclusive_sum((count + bm - 1) / bm);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  const uint64_t all = (uint64_t)total * ntiles;
  const uint64_t per = all / kXcds, rem = all % kXcds;
  const uint32_t x = bid % kXcds, idx = bid / kXcds;
  if (idx >= per + (x < rem ? 1 : 0)) return false;
  const uint64_t tile = x * per + min((uint64_t)x, rem) + idx;
  const uint32_t mt = __builtin_amdgcn_readfirstlane((uint32_t)(tile / ntiles));
  t->n = __builtin_amdgcn_readfirstlane((int)(tile % ntiles));
  uint32_t before = 0;
  for (int c = 0; c < groups; c += 64) {
    if (groups > 64) {
      begin = count = 0;
      if (c + lane < groups) group_range(off, c + lane, rows, &begin, &count);
      incl = wave_inclusive_sum((count + bm - 1) / bm);
    }
    const uint64_t hit = __ballot(before + (uint32_t)incl > mt);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int tiles = (count + bm - 1) / bm;
      t->g = c + l;
      t->begin = __builtin_amdgcn_readlane(begin, l);
      t->count = __builtin_amdgcn_readlane(count, l);
      t->m = mt - before - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles, l));
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// One operand tile in LDS, in 16-byte chunks (8 two-byte values).  KC: the
// contraction is contiguous in memory; R rows of BK values, whose chunks are
// permuted by the row so that the 8 rows a fragment read touches at once lie in
// different banks.  Else BK contraction steps of R contiguous values, read back
// with the transposing LDS load, whose 16 lanes take 32 bytes of 4 steps each:
// chunks are permuted in pairs by the step.
template <bool KC, int R, int BK>
struct LdsTile {
  static constexpr int kChunks = R * BK / 8;
  static constexpr int kPerRow = KC ? BK / 8 : R / 8;
  static __device__ __forceinline__ int swizzle(int line, int c) {
    if (KC) return BK == 32 ? c ^ ((line >> 2) & 3) : c ^ (line & 7);
    return c ^ ((line & 7) << 1);
  }
  // position of chunk c of a line (a row, or a contraction step)
  static __device__ __forceinline__ int pos(int line, int c) { return line * kPerRow + swizzle(line, c); }

  // the 8 contraction values k0 + 8 * (lane / 16) ... of row r0 + lane % 16
  static __device__ __forceinline__ s16x8 fragment(const i32x4* lds, int r0, int k0) {
    const int lane = threadIdx.x & 63;
    if (KC) {
      return __builtin_bit_cast(s16x8, lds[pos(r0 + (lane & 15), (k0 >> 3) + (lane >> 4))]);
    } else {
      typedef __attribute__((address_space(3))) s16x4* lds_p;
      const int step = k0 + (lane >> 4) * 8 + ((lane & 15) >> 2);
      const int c = (r0 >> 3) + ((lane & 3) >> 1);
      const char* base = reinterpret_cast<const char*>(lds) + (lane & 1) * 8;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(base + pos(step, c) * 16));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(base + pos(step + 4, c) * 16));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// 8 values of a two-byte matrix from (line, c * 8) on, zeros where the line or
// the column lies outside: lines of `ld` values at any 2-byte aligned address.
template <bool FLAT>
__device__ __forceinline__ i32x4 load_chunk(const uint16_t* base, uint64_t ld, int line, int lines, int col, int cols) {
  i32x4 v = {0, 0, 0, 0};
  if (line >= lines || col >= cols) return v;
  const uint16_t* p = base + (uint64_t)line * ld + col;
  const int left = cols - col;
  if (left >= 8) return FLAT ? *reinterpret_cast<const i32x4*>(p) : load16(p);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (j < left) w[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
  v[0] = w[0]; v[1] = w[1]; v[2] = w[2]; v[3] = w[3];
  return v;
}

// Four consecutive outputs of one row, those left of `cols`.
template <typename O>
struct Out4;
template <typename E>
struct __attribute__((packed, aligned(sizeof(E)))) Pack4 {
  E v[4];
};
template <typename O>
__device__ __forceinline__ void store4(O* row, int col, int cols, f32x4 v) {
  if (col + 4 <= cols) {
    Pack4<O> p;
#pragma unroll
    for (int i = 0; i < 4; i++) p.v[i] = (O)v[i];
    *reinterpret_cast<Pack4<O>*>(row + col) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (col + i < cols) row[col + i] = (O)v[i];
  }
}

}  // namespace
}  // namespace ciera
