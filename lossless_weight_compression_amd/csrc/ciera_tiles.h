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
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef __bf16 T;
  typedef bf16x8 V;
  static constexpr bool kScaled = false;
};
struct Fp16 {
  typedef _Float16 T;
  typedef f16x8 V;
  static constexpr bool kScaled = false;
};
struct Mx4 {  // 32 codes
  typedef i32x4 V;
  static constexpr bool kScaled = true;
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// 16 x 16 results over 128 steps: a lane's 32 codes and their scale, in the lowest byte.
__device__ __forceinline__ f32x4 mfma(i32x4 a, int scale_a, i32x4 b, int scale_b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                          i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, 0, scale_a, 0,
                                                          scale_b);
}
// 32 x 32 results over 64 steps, the scales in byte U.
template <int U>
__device__ __forceinline__ f32x16 mfma(i32x4 a, int scale_a, i32x4 b, int scale_b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                         i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, U, scale_a, U,
                                                         scale_b);
}

// 16 bytes at any 2-byte aligned address (the hardware splits what crosses a line).
struct __attribute__((packed, aligned(2))) Bytes16 {
  i32x4 v;
};
__device__ __forceinline__ i32x4 load16(const void* p) { return reinterpret_cast<const Bytes16*>(p)->v; }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
template <typename T>
__device__ __forceinline__ T read_lds(uint32_t at) {
  return *(__attribute__((address_space(3))) const T*)(uintptr_t)at;
}
// The transposing LDS load, twice: of every 16 lanes, lane i gets column i of the rows
// of 16 two-byte values that they address (4 lanes, 8 bytes each, to a row): 4 rows,
// and 4 more `next` bytes on.
__device__ __forceinline__ s16x8 read_transposed(uint32_t at, uint32_t next) {
  typedef __attribute__((address_space(3))) s16x4* lds_p;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(uintptr_t)at);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(uintptr_t)(at + next));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

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

// Sum of v over the lanes up to and including this one: within rows of 16 lanes,
// then each row's total added to the rows after it.
__device__ __forceinline__ int wave_inclusive_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from 1 lane below
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of the row below, to rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31, to rows 2 and 3
  return v;
}

// The row tiles (height BM) of all groups, numbered in order.  Each wave adds them
// up by itself, 64 groups at a time; up to 64 groups stay in registers.
struct GroupTile {
  int g, m, begin, count;  // tile m of group g: rows [begin + m * BM, begin + count)
};
template <int BM>
struct GroupTiles {
  const int32_t* off;
  int groups, rows;
  int begin, count, incl;  // of this lane's group in the chunk of 64 last looked at
  uint32_t total;

  __device__ __forceinline__ void chunk(int c) {
    const int g = c + (threadIdx.x & 63);
    begin = count = 0;
    if (g < groups) group_range(off, g, rows, &begin, &count);
    incl = wave_inclusive_sum((count + BM - 1) / BM);
  }
  __device__ __forceinline__ void init(const int32_t* o, int g, int r) {
    off = o;
    groups = g;
    rows = r;
    total = 0;
    for (int c = 0; c < groups; c += 64) {
      chunk(c);
      total += (uint32_t)__builtin_amdgcn_readlane(incl, 63);
    }
  }
  // row tile mt < total
  __device__ __forceinline__ GroupTile find(uint32_t mt) {
    uint32_t before = 0;
    int c = 0;
    if (groups > 64) {
      for (;; c += 64) {
        chunk(c);
        const uint32_t t = (uint32_t)__builtin_amdgcn_readlane(incl, 63);
        if (before + t > mt || c + 64 >= groups) break;
        before += t;
      }
    }
    const uint64_t hit = __ballot(before + (uint32_t)incl > mt);
    const int l = hit ? __builtin_ctzll(hit) : 0;
    GroupTile t;
    t.g = c + l;
    t.begin = __builtin_amdgcn_readlane(begin, l);
    t.count = __builtin_amdgcn_readlane(count, l);
    t.m = (int)(mt - before) - (__builtin_amdgcn_readlane(incl, l) - (t.count + BM - 1) / BM);
    return t;
  }
};

// Share of one of `all` equal tiles' lists: workgroups are dealt to the dies in
// turn, so each die gets one contiguous run of the tiles and its L2 holds few
// groups' operands at a time.  [*first, *first + *n) is die x's run.
__device__ __forceinline__ void die_run(uint64_t all, uint32_t x, uint64_t* first, uint32_t* n) {
  const uint64_t per = all / kXcds, rem = all % kXcds;
  *first = x * per + (x < rem ? x : rem);
  *n = (uint32_t)(per + (x < rem ? 1 : 0));
}

// f(0), f(1), ... with the number as a constant.
template <int I>
struct Int {
  static constexpr int v = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(Int<I>());
    each<N, I + 1>(f);
  }
}

// Row tile and column tile of workgroup `bid`, one tile each; false: beyond the
// last tile (the grid covers the largest possible number).  Up to 64 groups at a time, or four
// times 64 whose offsets are loaded at once and, up to 256 groups, once: what a workgroup with
// little work waits for first.
template <int BM>
__device__ __forceinline__ bool find_group_tile(const int32_t* off, int groups, int rows, int ntiles, uint32_t bid,
                                                GroupTile* t, int* n) {
  int begin[4], count[4], incl[4];
  uint32_t sums[4];
  auto chunks = [&](int c, auto four) {
    constexpr int N = decltype(four)::v;  // or one
    // behind the last group both ends are the last offset
    int from[N], to[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int g = c + i * 64 + (threadIdx.x & 63);
      from[i] = off[min(g, groups)];
      to[i] = off[min(g + 1, groups)];
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      begin[i] = count[i] = 0;
      if (i >= N) continue;
      begin[i] = min(max(from[i], 0), rows);
      count[i] = max(min(max(to[i], 0), rows) - begin[i], 0);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      sums[i] = incl[i] = 0;
      if (i >= N || c + i * 64 >= groups) continue;
      incl[i] = wave_inclusive_sum((count[i] + BM - 1) / BM);
      sums[i] = (uint32_t)__builtin_amdgcn_readlane(incl[i], 63);
    }
    return sums[0] + sums[1] + sums[2] + sums[3];
  };
  uint32_t total = 0;
  if (!off) total = (rows + BM - 1) / BM;
  else if (groups <= 64) total = chunks(0, Int<1>());
  else
    for (int c = 0; c < groups; c += 256) total += chunks(c, Int<4>());
  uint64_t first;
  uint32_t many;
  die_run((uint64_t)total * ntiles, bid % kXcds, &first, &many);
  if (bid / kXcds >= many) return false;
  const uint64_t tile = first + bid / kXcds;
  const uint32_t mt = (uint32_t)(tile / ntiles);
  *n = (int)(tile % ntiles);
  GroupTile r = {0, (int)mt, 0, rows};
  if (off) {
    uint32_t before = 0;
    int c = 0;
    if (groups > 256) {
      for (;; c += 256) {
        const uint32_t all = chunks(c, Int<4>());
        if (before + all > mt || c + 256 >= groups) break;
        before += all;
      }
    }
    // the chunk of 64 that it is in
    int i = 0, b = begin[0], k = count[0], up = incl[0];
#pragma unroll
    for (int j = 0; j < 3; j++) {
      const bool on = i == j && mt >= before + sums[j];
      before += on ? sums[j] : 0;
      i = on ? j + 1 : i;
      b = on ? begin[j + 1] : b;
      k = on ? count[j + 1] : k;
      up = on ? incl[j + 1] : up;
    }
    const uint64_t hit = __ballot(before + (uint32_t)up > mt);
    const int l = hit ? __builtin_ctzll(hit) : 0;
    r.g = c + i * 64 + l;
    r.begin = __builtin_amdgcn_readlane(b, l);
    r.count = __builtin_amdgcn_readlane(k, l);
    r.m = (int)(mt - before) - (__builtin_amdgcn_readlane(up, l) - (r.count + BM - 1) / BM);
  }
  *t = r;
  return true;
}

// v, as if computed anew here: what depends on it is not kept in registers across the
// main loop.
__device__ __forceinline__ int afresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
// LDS writes of this wave's lanes before, reads by others after (and the other way
// round): the LDS unit takes a wave's accesses in order, the compiler has to.
__device__ __forceinline__ void wave_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// One operand of a stage in LDS: R rows, 64 contraction steps of two bytes, in
// 16-byte chunks.  KC: the contraction is contiguous in memory, 8 chunks to a row; else
// R / 8 chunks to a contraction step, read back with the transposing load.
//
// A fragment is S rows, 16 or (4-bit operands, which are KC) 32.  COLS (the operand whose rows are the result's columns):
// they are taken in an order that gives a lane, which gets 4 of them together as results,
// 8 consecutive columns.
//
// The chunks of a line (a row, or a contraction step) are permuted by the line, so that
// what the lanes of one LDS cycle read lies in different banks: pieces of 4 contraction
// steps, or chunks of 16 lanes, which are not neighbours (0-3, 12-15, 20-23 and 24-27, and
// so on): with 32 rows to a fragment, even rows 0 2 12 14 20 22 24 26 and their odd
// neighbours need 8 different places.
template <bool KC, bool COLS, int S, int R = 256>
struct StageTile {
  static_assert(KC || S == 16, "32 rows are read back along the contraction only");
  static constexpr int kChunks = R * 8, kPerRow = KC ? 8 : R / 8;
  static __device__ __forceinline__ int swizzle(int line, int c) {
    const int k = (line & 3) | ((line >> 1) & 4);
    if (KC && S == 32) return c ^ (((line >> 1) & (COLS ? 1 : 3)) | (COLS ? (line >> 2) & 2 : 0) | ((line >> 2) & 4));
    if (KC) return c ^ (COLS ? k : line & 7);
    if (!COLS) return c ^ ((R == 64 ? line & 3 : k) << 1);
    return c ^ ((line & 3) << 2);
  }
  static __device__ __forceinline__ int pos(int line, int c) { return line * kPerRow + swizzle(line, c); }
  // the row of fragment 0 that this lane reads
  static __device__ __forceinline__ int first_row() {
    const int v = threadIdx.x & (S - 1);
    if (!COLS) return v;
    return S == 16 ? ((v & 12) << 1) + (v & 3) : (v & 16) + ((v >> 2) & 1) * 8 + ((v >> 3) & 1) * 4 + (v & 3);
  }
  // Where this lane reads fragment 0 of the rows from r0 on in the first part of the
  // stage (an address in LDS).  Other fragments and parts lie at that place with bits
  // flipped and a constant added, which costs no register each.  S = 16: a part is half
  // a stage, 8 steps of it to each 16 lanes.  S = 32: a part is 8 steps of each half of
  // the stage, one for each half of the wave.
  static __device__ __forceinline__ uint32_t place(const i32x4* lds, int r0) {
    const int lane = threadIdx.x & 63, p = lane & 3;
    if (KC) return lds_address(lds) + pos(r0 + first_row(), S == 16 ? lane >> 4 : (lane >> 5) * 4) * 16;
    const int step = (lane >> 4) * 8 + ((lane >> 2) & 3), c = COLS ? p : p >> 1, half = COLS ? 0 : p & 1;
    return lds_address(lds) + pos(step, r0 / 8 + c) * 16 + half * 8;
  }
  // GAP: COLS, from one pair of fragments to the next.
  template <int F, int PART, int GAP = 32>
  static __device__ __forceinline__ s16x8 fragment(uint32_t place) {
    constexpr int ROW = S == 32 ? F * 32 : COLS ? (F >> 1) * GAP + (F & 1) * 4 : F * 16;
    if constexpr (KC) return read_lds<s16x8>((place ^ (PART * (S == 16 ? 64 : 16))) + ROW * kPerRow * 16);
    constexpr int FLIP = ROW / 8 * 16, HALF = (ROW & 7) * 2;
    return read_transposed((place ^ FLIP) + PART * 32 * kPerRow * 16 + HALF, 4 * kPerRow * 16);
  }
};

// The first `left` of 8 two-byte values, zeros behind.  Loads that do not wait for each
// other: 13 groups of 1447 x 777, fp16, 2234 rows, 29.7 us for 30.9 with a branch to each,
// [N, K] 31.2 for 34.8, with 40000 rows 175 for 206.
__device__ __forceinline__ i32x4 load_some(const uint16_t* p, int left) {
  if (left >= 8) return load16(p);
  if (left <= 0) return i32x4{0, 0, 0, 0};
  // all at once, the last one again in place of those behind it
  uint32_t v[8], w[4];
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = p[min(j, left - 1)];
#pragma unroll
  for (int j = 0; j < 8; j += 2) w[j / 2] = (j < left ? v[j] : 0) | (j + 1 < left ? v[j + 1] << 16 : 0);
  return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// Consecutive outputs of one row, at any element.
template <typename E, int N>
struct __attribute__((packed, aligned(2))) Pack {
  E v[N];
};
template <typename O>
__device__ __forceinline__ void store4(O* row, int col, int cols, f32x4 v) {
  if (col + 4 <= cols) {
    Pack<O, 4> p;
#pragma unroll
    for (int i = 0; i < 4; i++) p.v[i] = (O)v[i];
    *reinterpret_cast<Pack<O, 4>*>(row + col) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (col + i < cols) row[col + i] = (O)v[i];
  }
}
// Up to 8 consecutive values of a row, zeros behind.
template <typename O>
__device__ __forceinline__ void load_row8(const O* at, int left, float* v) {
  if (left >= 8) {
    const Pack<O, 8> p = *reinterpret_cast<const Pack<O, 8>*>(at);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = (float)p.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = i < left ? (float)at[i] : 0.f;
  }
}
// 8 outputs: one store in two-byte types, two in fp32.
template <typename O>
__device__ __forceinline__ void store8(O* at, f32x4 lo, f32x4 hi) {
  constexpr int N = sizeof(O) == 2 ? 8 : 4;
  Pack<O, N> p[8 / N];
#pragma unroll
  for (int i = 0; i < 8; i++) p[i / N].v[i % N] = (O)(i < 4 ? lo[i & 3] : hi[i & 3]);
#pragma unroll
  for (int i = 0; i < 8 / N; i++) reinterpret_cast<Pack<O, N>*>(at)[i] = p[i];
}
// Up to 8.
template <typename O>
__device__ __forceinline__ void store_row8(O* at, int left, f32x4 lo, f32x4 hi) {
  if (left >= 8) {
    store8(at, lo, hi);
  } else {
    store4(at, 0, left, lo);
    store4(at, 4, left, hi);
  }
}

}  // namespace
}  // namespace ciera
