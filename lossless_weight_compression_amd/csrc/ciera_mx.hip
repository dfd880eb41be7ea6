// Microscaled 4-bit floating point: quantisation, its reverse, and the product
// of two 4-bit matrices.
//
// A block of 32 values v shares the scale 2^e, e = floor(log2(max |v|)) - 2 (the
// largest of the 4-bit magnitudes 0 .5 1 1.5 2 3 4 6 has exponent 2), kept as the
// byte e + 127 and never below 0; each value is the nearest magnitude to
// |v| 2^-e, ties to the even code, above 6 the 6 itself, with v's sign in bit 3.
#include "ciera.h"
#include "ciera_big.h"
#include "ciera_mid.h"
#include "ciera_ops_internal.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Scale byte of a block from the exponent field (of fp32) of its largest magnitude:
// the field less 2.  Infinity and NaN have the field 255, whose byte means NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t field) {
  return field == 255 ? 255u : field > 2 ? field - 2 : 0u;
}
// 2^(byte - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// An input type.  A word is what 32 bits of memory hold: kPer values.  Magnitudes are
// compared as integers: that orders them, infinity above all numbers and NaN above it.
// code2: two values to two codes, into byte SEL of `old`; the conversion divides by
// the scale, rounds to nearest even and stops at 6.
template <typename V2>
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(V2, a), __builtin_bit_cast(V2, b)));
}
struct Bf16In {
  typedef uint16_t T;
  static constexpr int kPer = 2;
  static __device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & 0x7fff7fffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max_halves<u16x2>(a, b); }
  static __device__ __forceinline__ uint32_t field(uint32_t m) { return m >> 7; }  // m: one value's magnitude
  template <int SEL>
  static __device__ __forceinline__ uint32_t code2(uint32_t old, uint32_t pair, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), s, SEL);
  }
};
struct Fp16In {
  typedef uint16_t T;
  static constexpr int kPer = 2;
  static __device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & 0x7fff7fffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max_halves<u16x2>(a, b); }
  static __device__ __forceinline__ uint32_t field(uint32_t m) {
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)m)) >> 23;
  }
  template <int SEL>
  static __device__ __forceinline__ uint32_t code2(uint32_t old, uint32_t pair, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, pair), s, SEL);
  }
};
struct Fp32In {
  typedef uint32_t T;
  static constexpr int kPer = 1;
  static __device__ __forceinline__ uint32_t magnitude(uint32_t w) { return w & 0x7fffffffu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t field(uint32_t m) { return m >> 23; }
  template <int SEL>
  static __device__ __forceinline__ uint32_t code2(uint32_t old, uint32_t lo, uint32_t hi, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi), s,
                                                    SEL);
  }
};

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

// Largest magnitude of N words of one block's values, as one value.
template <typename I, int N>
__device__ __forceinline__ uint32_t largest(const uint32_t* w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; i++) m = I::larger(m, I::magnitude(w[i]));
  return I::kPer == 2 ? max(m & 0xffffu, m >> 16) : m;
}
// 8 values to 8 codes, the first in the low nibble.  A block with infinities or NaN
// holds zeros behind its NaN scale.
template <typename I>
__device__ __forceinline__ uint32_t encode8(const uint32_t* w, uint32_t byte) {
  const float s = scale_value(byte);
  uint32_t r;
  if constexpr (I::kPer == 2) {
    r = I::template code2<0>(0, w[0], s);
    r = I::template code2<1>(r, w[1], s);
    r = I::template code2<2>(r, w[2], s);
    r = I::template code2<3>(r, w[3], s);
  } else {
    r = I::template code2<0>(0, w[0], w[1], s);
    r = I::template code2<1>(r, w[2], w[3], s);
    r = I::template code2<2>(r, w[4], w[5], s);
    r = I::template code2<3>(r, w[6], w[7], s);
  }
  return byte == 255 ? 0 : r;
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

// Blocks along the rows of x: 4 lanes to a block, 8 values each.
template <typename I>
__global__ __launch_bounds__(256) void mx_quantize_rows(MxQuantArgs a, RowPass pass) {
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRun;
  for (uint64_t s0 = first_segment(); s0 < pass.total; s0 += step) {
    uint32_t w[kRun][8 / I::kPer], chunk[kRun];
    uint64_t line[kRun];
    bool on[kRun];
#pragma unroll
    for (int i = 0; i < kRun; i++) {
      on[i] = pass.locate(s0 + i, &line[i], &chunk[i]);
      const uint64_t g = a.groups == 1 ? 0 : pass.quotient(line[i], a.rows), r = line[i] - g * a.rows;
      const typename I::T* p = static_cast<const typename I::T*>(a.x) + g * a.gsx + r * a.ldx + chunk[i] * 8;
      load8<I>(p, on[i] ? a.cols - (int)chunk[i] * 8 : 0, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kRun; i++) {
      uint32_t m = largest<I, 8 / I::kPer>(w[i]);
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));  // lane ^ 1
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));  // lane ^ 2
      if (!on[i]) continue;
      const uint32_t byte = scale_byte(I::field(m));
      const uint64_t o = line[i] * pass.chunks + chunk[i];
      reinterpret_cast<uint32_t*>(a.codes)[o] = encode8<I>(w[i], byte);
      if ((chunk[i] & 3) == 0) a.scales[o / 4] = (uint8_t)byte;
    }
  }
}

// Blocks down the columns of x: row c of the result is column c of x.  A workgroup
// takes 8 blocks (256 rows of x), one to a wave, of 64 words' columns: a wave reads 256
// bytes of each row, a lane holds the 32 values of its one or two columns.  The codes
// go through LDS, so that 8 lanes write the 128 bytes of 8 blocks of one column.  LINES:
// what a wave reads of a row is whole lines, which nobody reads again (64 x 2048 x 1024,
// bf16, read past the caches 58 us, 5.9 TB/s, for 65; where rows share lines 49 for 44).
template <typename I, bool LINES>
__global__ __launch_bounds__(512) void mx_quantize_cols(MxQuantArgs a) {
  constexpr int C = 64 * I::kPer;  // columns
  __shared__ i32x4 codes[8 * C];
  __shared__ uint8_t scales[8 * C];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t blocks = (uint32_t)((a.rows + (int)kMxColsPad - 1) / (int)kMxColsPad) * (kMxColsPad / kMxBlock);
  const uint32_t btiles = (blocks + 7) / 8, ctiles = (a.cols + C - 1) / C;
  const uint64_t all = (uint64_t)btiles * ctiles * a.groups;
  for (uint64_t t = blockIdx.x; t < all; t += gridDim.x) {
    const uint64_t g = t / ((uint64_t)btiles * ctiles);
    const uint32_t b0 = (uint32_t)(t / ctiles % btiles) * 8;
    const int c0 = (int)(t % ctiles) * C;
    const int b = b0 + wave, c = c0 + lane * I::kPer;
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; j++) w[j] = 0;
    const int rows = min(max(a.rows - b * 32, 0), 32);
    if (c < a.cols) {
      // a lane whose second column lies outside reads the word before and drops its first half
      const bool half = I::kPer == 2 && c + 1 == a.cols && a.cols > 1, one = I::kPer == 2 && a.cols == 1;
      const typename I::T* p =
          static_cast<const typename I::T*>(a.x) + g * a.gsx + (uint64_t)b * 32 * a.ldx + c - (half ? 1 : 0);
      auto word = [&](int j) -> uint32_t {
        const typename I::T* q = p + (uint64_t)j * a.ldx;
        if (LINES) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q));
        if (one) return *q;
        return reinterpret_cast<const Pack<uint16_t, 2>*>(q)->v[0] |
               (uint32_t) reinterpret_cast<const Pack<uint16_t, 2>*>(q)->v[1] << 16;
      };
      if (rows == 32) {
#pragma unroll
        for (int j = 0; j < 32; j++) w[j] = word(j);
      } else {
#pragma unroll
        for (int j = 0; j < 32; j++)
          if (j < rows) w[j] = word(j);
      }
      if (half) {
#pragma unroll
        for (int j = 0; j < 32; j++) w[j] >>= 16;
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; j++) m = I::larger(m, I::magnitude(w[j]));
#pragma unroll
    for (int h = 0; h < I::kPer; h++) {
      const uint32_t byte = scale_byte(I::field(I::kPer == 1 ? m : h ? m >> 16 : m & 0xffffu));
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        uint32_t v[8 / I::kPer];
#pragma unroll
        for (int j = 0; j < 8 / I::kPer; j++)  // of two-byte types, the pairs of this column
          v[j] = I::kPer == 1 ? w[i * 8 + j]
                              : __builtin_amdgcn_perm(w[(i * 8 + 2 * j + 1) & 31], w[(i * 8 + 2 * j) & 31],
                                                      h ? 0x07060302u : 0x05040100u);
        q[i] = encode8<I>(v, byte);
      }
      const int col = lane * I::kPer + h;
      codes[col * 8 + (wave ^ (lane & 7))] = i32x4{(int)q[0], (int)q[1], (int)q[2], (int)q[3]};
      scales[col * 8 + wave] = (uint8_t)byte;
    }
    __syncthreads();
    const uint64_t row0 = g * a.cols + c0;  // of the result
#pragma unroll
    for (int i = 0; i < C * 8 / 512; i++) {
      const int p = i * 512 + tid, col = p >> 3, k = p & 7;
      if (c0 + col < a.cols && b0 + k < blocks)
        reinterpret_cast<i32x4*>(a.codes)[(row0 + col) * blocks + b0 + k] = codes[col * 8 + (k ^ (col / I::kPer & 7))];
    }
    for (int p = tid; p < C * 2; p += 512) {  // 4 scales at a time
      const int col = p >> 1, k = (p & 1) * 4;
      if (c0 + col < a.cols && b0 + k < blocks)
        *reinterpret_cast<uint32_t*>(a.scales + (row0 + col) * blocks + b0 + k) =
            *reinterpret_cast<const uint32_t*>(scales + col * 8 + k);
    }
    __syncthreads();
  }
}

template <typename O>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, Pack<O, 8>* out) {
  const float s = scale_value(byte), nan = __builtin_nanf("");
  const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
  const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
  const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  const float v[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
#pragma unroll
  for (int j = 0; j < 8; j++) out->v[j] = (O)(byte == 255 ? nan : v[j]);
}

// Every value is exact in bf16: the conversion goes there at once.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, Pack<__bf16, 8>* out) {
  const float s = scale_value(byte);
  uint32_t v[4] = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
#pragma unroll
  for (int j = 0; j < 4; j++) v[j] = byte == 255 ? 0x7fc07fc0u : v[j];
  __builtin_memcpy(out, v, 16);
}

// Rows without padding or gaps, one after another: every chunk of codes lies where its
// values go.  A workgroup takes 1024 consecutive chunks, 4 loads to a lane under way.
template <typename O>
__global__ __launch_bounds__(256) void mx_dequantize_flat(const uint32_t* codes, const uint8_t* scales, O* out,
                                                          uint64_t chunks) {
  for (uint64_t b = blockIdx.x; b * 1024 < chunks; b += gridDim.x) {
    const uint64_t i = b * 1024 + threadIdx.x;
    uint32_t w[4], byte[4];
    if (b * 1024 + 1024 <= chunks) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        w[j] = codes[i + j * 256];
        byte[j] = scales[(i + j * 256) / 4];
      }
#pragma unroll
      for (int j = 0; j < 4; j++) decode8(w[j], byte[j], reinterpret_cast<Pack<O, 8>*>(out) + i + j * 256);
    } else {
      for (uint64_t k = i; k < chunks; k += 256)
        decode8(codes[k], scales[k / 4], reinterpret_cast<Pack<O, 8>*>(out) + k);
    }
  }
}

template <typename O>
__global__ __launch_bounds__(256) void mx_dequantize(MxDequantArgs a, RowPass pass) {
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRun;
  for (uint64_t s0 = first_segment(); s0 < pass.total; s0 += step) {
    uint32_t w[kRun], byte[kRun], chunk[kRun];
    uint64_t line[kRun];
    int left[kRun];
#pragma unroll
    for (int i = 0; i < kRun; i++) {
      const bool on = pass.locate(s0 + i, &line[i], &chunk[i]);
      left[i] = on ? a.cols - (int)chunk[i] * 8 : 0;
      const uint64_t o = line[i] * pass.chunks + chunk[i];
      w[i] = left[i] > 0 ? reinterpret_cast<const uint32_t*>(a.codes)[o] : 0;
      byte[i] = left[i] > 0 ? a.scales[o / 4] : 0;
    }
#pragma unroll
    for (int i = 0; i < kRun; i++) {
      if (left[i] <= 0) continue;
      const uint64_t g = a.groups == 1 ? 0 : pass.quotient(line[i], a.rows), r = line[i] - g * a.rows;
      O* p = static_cast<O*>(a.out) + g * a.gso + r * a.ldo + chunk[i] * 8;
      Pack<O, 8> v;
      decode8(w[i], byte[i], &v);
      if (left[i] >= 8) {
        *reinterpret_cast<Pack<O, 8>*>(p) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (j < left[i]) p[j] = v.v[j];
      }
    }
  }
}

// out = a b^T on the rows of every group.  In units of two bytes (4 codes) the operands
// look like two-byte ones.
template <typename O>
__global__ __launch_bounds__(256, 2) void mx_mm_mid(MxMmArgs a) {
  constexpr int BM = 64;
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + 127) / 128, blockIdx.x, &t, &tn)) return;
  const int n0 = tn * 128, units = a.kp / 4;
  const uint32_t srow = a.kp / 32;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM, brow = (uint64_t)t.g * a.n + n0;
  mid_tile<Mx4, true, true, O, BM, 1>(reinterpret_cast<const uint16_t*>(a.a) + row * units, units, t.count - t.m * BM,
                                   reinterpret_cast<const uint16_t*>(a.b) + brow * units, units, a.n - n0, units,
                                   static_cast<O*>(a.out) + row * a.ldo + n0, a.ldo, a.sa + row * srow, a.sb + brow * srow,
                                   srow);
}

// Large products: 256 x 256 tiles, 256 codes of every row at a time.
template <typename O>
__global__ __launch_bounds__(512) void mx_mm_big(MxMmArgs a) {
  typedef BigTiles<Mx4, true, true, O> Big;
  __shared__ i32x4 lds[Big::kLds];
  GroupTiles<256> tiles;
  tiles.init(a.offsets, a.groups, a.rows);
  const uint32_t nt = (a.n + 255) / 256;
  TileList list;
  list.init((uint64_t)tiles.total * nt);
  Big big;
  big.init(lds);
  const int units = a.kp / 4;
  const uint32_t srow = a.kp / 32;
  O* out;
  int om, on, half = 0;
  auto start = [&](uint32_t i) {
    uint64_t tile;
    int r0, rows;
    if (!list.get(i, &tile, &r0, &rows)) return false;
    const GroupTile t = tiles.find((uint32_t)(tile / nt));
    const int n0 = (int)(tile % nt) * 256;
    const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 256 + r0, brow = (uint64_t)t.g * a.n + n0;
    om = min(t.count - t.m * 256 - r0, rows);
    on = a.n - n0;
    if (om <= 0) return false;
    out = static_cast<O*>(a.out) + row * a.ldo + n0;
    big.scales(a.sa + row * srow, om, a.sb + brow * srow, on, srow);
    big.start(reinterpret_cast<const uint16_t*>(a.a) + row * units, units, om,
              reinterpret_cast<const uint16_t*>(a.b) + brow * units, units, on, units, half);
    return true;
  };
  if (!start(0)) return;
  for (uint32_t i = 1;; i++) {
    big.stages(om, units, &half);
    O* done = out;
    const int dm = om, dn = on;
    const bool more = start(i);
    big.finish(done, a.ldo, dm, dn);
    if (!more) return;
  }
}

// Few rows to a group: 16 rows and 16 columns to a workgroup.  Its 4 waves take
// runs of 512 codes of every row in turn, from memory into registers: a lane 4 blocks
// and the word of their scales; their sums are joined through LDS in order.
constexpr int kMxThinWaves = 4;

template <typename O>
__global__ __launch_bounds__(256) void mx_mm_thin(MxMmArgs a) {
  constexpr int BN = 16, LD = BN + 4;
  __shared__ __attribute__((aligned(16))) float part[kMxThinWaves * 16 * LD];
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16, q = lane >> 4;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  const int blocks = a.kp / 32;
  const uint64_t wr = (uint64_t)t.g * a.n + n0 + min(lane & 15, left - 1);
  const i32x4* pw = reinterpret_cast<const i32x4*>(a.b) + wr * blocks;
  const uint8_t* psw = a.sb + wr * blocks;
  const uint64_t xr = row + min(lane & 15, rows - 1);
  const i32x4* px = reinterpret_cast<const i32x4*>(a.a) + xr * blocks;
  const uint8_t* psx = a.sa + xr * blocks;
  f32x4 acc = {0, 0, 0, 0};
  for (int b0 = wave * 16; b0 < blocks; b0 += kMxThinWaves * 16) {
    const int b = b0 + q * 4;  // rows hold multiples of 4 blocks: a lane's run is in or out
    i32x4 w[4], x[4];
    uint32_t sw = 0, sx = 0;
#pragma unroll
    for (int u = 0; u < 4; u++) w[u] = x[u] = i32x4{0, 0, 0, 0};
    if (b < blocks) {
#pragma unroll
      for (int u = 0; u < 4; u++) {
        w[u] = pw[b + u];
        x[u] = px[b + u];
      }
      sw = *reinterpret_cast<const uint32_t*>(psw + b);
      sx = *reinterpret_cast<const uint32_t*>(psx + b);
    }
#pragma unroll
    for (int u = 0; u < 4; u++) acc = mfma(w[u], (int)(sw >> (8 * u)), x[u], (int)(sx >> (8 * u)), acc);
  }
  float* mine = part + (wave * 16 + (lane & 15)) * LD + (lane >> 4) * 4;
  *reinterpret_cast<f32x4*>(mine) = acc;
  __syncthreads();
  O* out = static_cast<O*>(a.out) + row * a.ldo + n0;
  for (int p = threadIdx.x; p < 16 * BN / 4; p += kMxThinWaves * 64) {
    const int m = p / (BN / 4), c = p % (BN / 4) * 4;
    if (m >= rows || c >= left) continue;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kMxThinWaves; w++) v += *reinterpret_cast<const f32x4*>(part + (w * 16 + m) * LD + c);
    store4(out + (uint64_t)m * a.ldo, c, left, v);
  }
}

// Workgroups of a pass; beyond the limit each takes several parts in turn.
uint32_t pass_grid(uint64_t parts, uint64_t limit) { return (uint32_t)(parts < limit ? parts : limit); }
uint32_t row_grid(const RowPass& p) { return pass_grid((p.total + 4 * kRun - 1) / (4 * kRun), 1 << 20); }

template <typename O>
hipError_t run_mx_mm(const MxMmArgs& a, hipStream_t s) {
  // By rows to a group on average; 64 experts of 2048 x 1024, us, the same operands from
  // call to call (at 1024 rows the large kernel takes 85, with operands from memory 125).
  // Where 64 x 128 tiles leave most of the card idle the thin kernel wins up to 64 rows (one
  // matrix 7168 x 2048, 24 rows 8.1 for 16.7, 64 rows 11.1 for 17.7; 1 token over 8 experts
  // 8 for 18):
  //   rows        4    8   16   24   64  100  128  160  200  256
  //   thin       18   21   21
  //   64 rows    14   15   19   19   20   29   32   36   44   52
  //   256 x 256                                39   38   38   39
  const int64_t rows = a.rows, groups = a.groups;
  const uint64_t mid = max_row_tiles(rows, groups, 64) * ((a.n + 127) / 128);
  const uint64_t big = max_row_tiles(rows, groups, 256) * ((a.n + 255) / 256);
  dim3 grid;
  if ((rows <= 16 * groups && mid < kUnits) || (rows <= 64 * groups && mid < kUnits / 4)) {
    if (hipError_t e = tile_grid(max_row_tiles(rows, groups, 16) * ((a.n + 15) / 16), 256, &grid)) return e;
    mx_mm_thin<O><<<grid, dim3(256), 0, s>>>(a);
  } else if (a.kp && rows >= 192 * groups && big >= kUnits / 2 && short_stride(a.kp / 4)) {
    mx_mm_big<O><<<dim3(kUnits), dim3(512), 0, s>>>(a);
  } else {
    if (hipError_t e = tile_grid(mid, 256, &grid)) return e;
    mx_mm_mid<O><<<grid, dim3(256), 0, s>>>(a);
  }
  return hipGetLastError();
}

template <bool LINES>
void quantize_cols(int dtype, dim3 grid, const MxQuantArgs& a, hipStream_t s) {
  if (dtype == CIERA_BF16) mx_quantize_cols<Bf16In, LINES><<<grid, dim3(512), 0, s>>>(a);
  else if (dtype == CIERA_FP16) mx_quantize_cols<Fp16In, LINES><<<grid, dim3(512), 0, s>>>(a);
  else mx_quantize_cols<Fp32In, LINES><<<grid, dim3(512), 0, s>>>(a);
}

}  // namespace

hipError_t launch_mx_quantize(int dtype, int axis, const MxQuantArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  if (axis) {
    // a stack without gaps is one matrix
    MxQuantArgs f = a;
    if (a.gsx == (uint64_t)a.rows * a.ldx && (uint64_t)a.rows * a.groups < (1u << 30)) {
      f.rows = a.rows * a.groups;
      f.groups = 1;
    }
    const RowPass pass(f.groups, f.rows, f.cols);
    const dim3 grid(row_grid(pass));
    if (dtype == CIERA_BF16) mx_quantize_rows<Bf16In><<<grid, dim3(256), 0, s>>>(f, pass);
    else if (dtype == CIERA_FP16) mx_quantize_rows<Fp16In><<<grid, dim3(256), 0, s>>>(f, pass);
    else mx_quantize_rows<Fp32In><<<grid, dim3(256), 0, s>>>(f, pass);
  } else {
    const uint64_t btiles = ((uint64_t)a.rows + 255) / 256, cols = dtype == CIERA_FP32 ? 64 : 128;
    const dim3 grid(pass_grid(btiles * ((a.cols + cols - 1) / cols) * a.groups, 1 << 20));
    const uint64_t line = dtype == CIERA_FP32 ? 32 : 64;  // values
    if (a.cols % line == 0 && a.ldx % line == 0 && a.gsx % line == 0 && reinterpret_cast<uintptr_t>(a.x) % 128 == 0)
      quantize_cols<true>(dtype, grid, a, s);
    else
      quantize_cols<false>(dtype, grid, a, s);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(int dtype, const MxDequantArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  MxDequantArgs f = a;
  if (a.gso == (uint64_t)a.rows * a.ldo && (uint64_t)a.rows * a.groups < (1u << 30)) {
    f.rows = a.rows * a.groups;
    f.groups = 1;
  }
  if (f.groups == 1 && f.cols % kMxColsPad == 0 && (f.rows == 1 || f.ldo == (uint64_t)f.cols)) {
    const uint64_t chunks = (uint64_t)f.rows * f.cols / 8;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(f.codes);
    const dim3 grid(pass_grid((chunks + 1023) / 1024, 1 << 20));
    if (dtype == CIERA_BF16) mx_dequantize_flat<<<grid, dim3(256), 0, s>>>(codes, f.scales, (__bf16*)f.out, chunks);
    else if (dtype == CIERA_FP16) mx_dequantize_flat<<<grid, dim3(256), 0, s>>>(codes, f.scales, (_Float16*)f.out, chunks);
    else mx_dequantize_flat<<<grid, dim3(256), 0, s>>>(codes, f.scales, (float*)f.out, chunks);
    return hipGetLastError();
  }
  const RowPass pass(f.groups, f.rows, f.cols);
  const dim3 grid(row_grid(pass));
  if (dtype == CIERA_BF16) mx_dequantize<__bf16><<<grid, dim3(256), 0, s>>>(f, pass);
  else if (dtype == CIERA_FP16) mx_dequantize<_Float16><<<grid, dim3(256), 0, s>>>(f, pass);
  else mx_dequantize<float><<<grid, dim3(256), 0, s>>>(f, pass);
  return hipGetLastError();
}

hipError_t launch_mx_mm(int out_dtype, const MxMmArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  if (out_dtype == CIERA_BF16) return run_mx_mm<__bf16>(a, s);
  if (out_dtype == CIERA_FP16) return run_mx_mm<_Float16>(a, s);
  return run_mx_mm<float>(a, s);
}

}  // namespace ciera
