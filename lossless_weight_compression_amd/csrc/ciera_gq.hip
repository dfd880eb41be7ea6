// 4-bit integer weights with group scales: quantisation and its reverse.
//
// A block of 32, 64 or 128 values v of a row shares a scale s and a zero z (0 to 15, 8 where
// none are kept): code q stands for s (q - z).  With zeros s spreads the 16 codes over the
// block's range, 0 in it: s = (hi - lo) (1 / 15), z = rint(-lo / s), q = rint(v / s) + z, both
// clamped to 0 ... 15; without, s = max |v| (1 / 7).  The product with the rounded 1 / 15 is what
// elementary tensor operations make of a division by 15, and gives their scales: 7 in 100000 fp16
// and 1 in 100000 bf16 ones, whose quotient lies within 2^-23 of the middle of two scales, are the
// other of the two, 0.5001 steps off the quotient for 0.5.
#include "ciera.h"
#include "ciera_gq.h"
#include "ciera_ops_internal.h"
#include "ciera_rows.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// s rounded to the scales' type, its bits; a scale below 2^-126 becomes 0.
__device__ __forceinline__ uint32_t scale_bits(float s, uint32_t half) {
  if (half) return __builtin_bit_cast(uint16_t, (_Float16)s);
  const uint32_t b = __builtin_bit_cast(uint16_t, (__bf16)s);
  return b < 0x80u ? 0u : b;
}

// v / s rounded to nearest, from r = 1 / s rounded: the quotient of the remainder corrects
// the product (exact remainder, one rounding).
__device__ __forceinline__ float quotient(float v, float s, float r) {
  const float q = v * r;
  return __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q);
}

struct BlockScale {
  uint32_t bits, zero;  // as stored
  float s, r;
  bool bad;
  // of a block with the smallest and the largest value, or (symmetric) the largest magnitude
  // in hi; not finite where one of its values is not
  __device__ __forceinline__ BlockScale(float lo, float hi, bool zeros, uint32_t half) {
    const float range = zeros ? (hi - lo) * (1.f / 15.f) : hi * (1.f / 7.f);
    bits = scale_bits(range, half);
    s = scale_of(bits, half);
    bad = !(s < __builtin_inff());
    if (bad) {
      bits = half ? 0x7e00u : 0x7fc0u;
      s = 0.f;
    }
    r = s > 0.f ? 1.f / s : 0.f;
    zero = bad ? 0u : zeros ? (uint32_t)fminf(fmaxf(__builtin_rintf(quotient(-lo, s, r)), 0.f), 15.f) : 8u;
  }
  // Quotients stay far below 2^22, so adding 1.5 2^23 rounds to the nearest integer, ties to
  // even, in the sum's low bits.
  __device__ __forceinline__ uint32_t code(float v) const {
    constexpr float kRound = 12582912.f;
    const int n = __builtin_bit_cast(int, quotient(v, s, r) + kRound) - __builtin_bit_cast(int, kRound) + (int)zero;
    return (uint32_t)min(max(n, 0), 15);
  }
};

// An input type.  A word is what 32 bits of memory hold: kPer values.  Extents are found in
// the values' bits, all of a word at once: as signed numbers the largest is that of the
// largest value, if one is positive, as unsigned ones that of the smallest, if one is
// negative.  Infinities and NaN come out on top of both.
template <typename V2>
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(V2, a), __builtin_bit_cast(V2, b)));
}
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t s16x2 __attribute__((ext_vector_type(2)));
struct GqTwo {
  typedef uint16_t T;
  static constexpr int kPer = 2;
  static constexpr uint32_t kMagnitudes = 0x7fff7fffu;
  static __device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) { return max_halves<s16x2>(a, b); }
  static __device__ __forceinline__ uint32_t largest_bits(uint32_t a, uint32_t b) { return max_halves<u16x2>(a, b); }
  static __device__ __forceinline__ uint32_t half(uint32_t w, int h) { return h ? w >> 16 : w & 0xffffu; }
};
struct GqBf16 : GqTwo {
  static __device__ __forceinline__ float number(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
  static __device__ __forceinline__ float value(const uint32_t* w, int j) {
    return __builtin_bit_cast(float, j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};
struct GqFp16 : GqTwo {
  static __device__ __forceinline__ float number(uint32_t bits) { return (float)__builtin_bit_cast(_Float16, (uint16_t)bits); }
  static __device__ __forceinline__ float value(const uint32_t* w, int j) { return number(half(w[j / 2], j & 1)); }
};
struct GqFp32 {
  typedef uint32_t T;
  static constexpr int kPer = 1;
  static constexpr uint32_t kMagnitudes = 0x7fffffffu;
  static __device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) { return (uint32_t)max((int)a, (int)b); }
  static __device__ __forceinline__ uint32_t largest_bits(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t half(uint32_t w, int) { return w; }
  static __device__ __forceinline__ float number(uint32_t bits) { return __builtin_bit_cast(float, bits); }
  static __device__ __forceinline__ float value(const uint32_t* w, int j) { return number(w[j]); }
};

// The largest and the smallest value of a block so far, with 0 (symmetric: the largest
// magnitude): bits, of each half of the words on its own.
template <typename I>
struct Extent {
  uint32_t top = 0, low = 0;
  __device__ __forceinline__ void add(uint32_t w, bool zeros) {
    if (zeros) {
      top = I::largest(top, w);
      low = I::largest_bits(low, w);
    } else {
      top = I::largest(top, w & I::kMagnitudes);
    }
  }
  __device__ __forceinline__ void join(uint32_t t, uint32_t l) {
    top = I::largest(top, t);
    low = I::largest_bits(low, l);
  }
  template <int CTRL>
  __device__ __forceinline__ void across() {  // lanes
    join((uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, CTRL, 0xf, 0xf, false),
         (uint32_t)__builtin_amdgcn_update_dpp(0, (int)low, CTRL, 0xf, 0xf, false));
  }
  __device__ __forceinline__ void join_halves() { join(top >> 16 | top << 16, low >> 16 | low << 16); }
  // of the values in half h of the words; a NaN counts as an infinity
  __device__ __forceinline__ float hi(int h) const { return finite_or_inf(I::number(I::half(top, h)), 1.f); }
  __device__ __forceinline__ float lo(int h) const {
    const float v = I::number(I::half(low, h));
    return finite_or_inf(v > 0.f ? 0.f : v, -1.f);
  }
  static __device__ __forceinline__ float finite_or_inf(float v, float sign) {
    return v == v ? v : sign * __builtin_inff();
  }
};

// 8 values to a word of codes.
template <typename F>
__device__ __forceinline__ uint32_t codes8(F value, const BlockScale& b) {
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) c |= b.code(value(j)) << (8 * (j & 3) + (j & 4));
  return b.bad ? 0 : c;
}
// Word c of a row's values in the order they are stored.
__device__ __forceinline__ uint32_t stored(uint32_t c) { return (c & ~15u) | (c & 3) << 2 | (c >> 2 & 3); }

// Blocks along the rows of x: BLOCK / 8 lanes to a block, 8 values each.
template <typename I, int BLOCK>
__global__ __launch_bounds__(256) void gq_quantize_rows(GqQuantArgs a, RowPass pass) {
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRun;
  const bool zeros = a.zeros != nullptr;
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
      Extent<I> e;
#pragma unroll
      for (int j = 0; j < 8 / I::kPer; j++) e.add(w[i][j], zeros);
      if (I::kPer == 2) e.join_halves();
      e.template across<0xb1>();                       // lane ^ 1
      e.template across<0x4e>();                       // lane ^ 2
      if (BLOCK >= 64) e.template across<0x141>();     // 7 - lane of 8
      if (BLOCK >= 128) e.template across<0x140>();    // 15 - lane of 16
      if (!on[i]) continue;
      const BlockScale b(e.lo(0), e.hi(0), zeros, a.half);
      reinterpret_cast<uint32_t*>(a.codes)[line[i] * pass.chunks + stored(chunk[i])] =
          codes8([&](int j) { return I::value(w[i], j); }, b);
      if (chunk[i] % (BLOCK / 8) == 0) {
        const uint64_t o = line[i] * (pass.chunks / (BLOCK / 8)) + chunk[i] / (BLOCK / 8);
        a.scales[o] = (uint16_t)b.bits;
        if (zeros) a.zeros[o] = (uint8_t)b.zero;
      }
    }
  }
}

// Blocks down the columns of x: row c of the result is column c of x.  A workgroup takes 256
// rows of x, 32 to a wave, of 64 words' columns: a wave reads 256 bytes of each row, a lane
// holds the 32 values of its one or two columns.  The waves of one block exchange their
// extents, and the codes go through LDS, so that 8 lanes write the 128 bytes of one column.
// LINES: what a wave reads of a row is whole lines, which nobody reads again.  64 x 2048 x 1024
// bf16, blocks of 128: 76 us, 4.4 TB/s, of which 12 vector instructions a value are a good part
// (extents value by value in fp32, two loads to a word: 209).
template <typename I, int BLOCK, bool LINES>
__global__ __launch_bounds__(512) void gq_quantize_cols(GqQuantArgs a) {
  constexpr int C = 64 * I::kPer, PER = BLOCK / 32;  // columns; waves to a block
  __shared__ i32x4 codes[8 * C];
  __shared__ uint2 extents[BLOCK > 32 ? 8 : 1][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool zeros = a.zeros != nullptr;
  const uint32_t words = (uint32_t)((a.rows + (int)kMxColsPad - 1) / (int)kMxColsPad) * (kMxColsPad / 8);  // of a result's row
  const uint32_t btiles = (words + 31) / 32, ctiles = (a.cols + C - 1) / C;
  const uint64_t all = (uint64_t)btiles * ctiles * a.groups;
  for (uint64_t t = blockIdx.x; t < all; t += gridDim.x) {
    const uint64_t g = t / ((uint64_t)btiles * ctiles);
    const uint32_t k0 = (uint32_t)(t / ctiles % btiles) * 256;
    const int c0 = (int)(t % ctiles) * C, c = c0 + lane * I::kPer, r0 = (int)k0 + wave * 32;
    const int rows = min(max(a.rows - r0, 0), 32);
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; j++) w[j] = 0;
    if (c < a.cols) {
      // a lane whose second column lies outside reads the word before and drops its first half
      const bool half = I::kPer == 2 && c + 1 == a.cols && a.cols > 1, one = I::kPer == 2 && a.cols == 1;
      const typename I::T* p = static_cast<const typename I::T*>(a.x) + g * a.gsx + (uint64_t)r0 * a.ldx + c - (half ? 1 : 0);
      auto word = [&](int j) -> uint32_t {
        const typename I::T* at = p + (uint64_t)j * a.ldx;
        if (LINES) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(at));
        if (one) return *at;
        return reinterpret_cast<const Pack<uint32_t, 1>*>(at)->v[0];
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
    Extent<I> e;
#pragma unroll
    for (int j = 0; j < 32; j++) e.add(w[j], zeros);
    if constexpr (BLOCK > 32) {
      extents[wave][lane] = make_uint2(e.top, e.low);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < PER; v++) {
        const uint2 o = extents[wave / PER * PER + v][lane];
        e.join(o.x, o.y);
      }
    }
#pragma unroll
    for (int h = 0; h < I::kPer; h++) {
      const BlockScale b(e.lo(h), e.hi(h), zeros, a.half);
      uint32_t* mine = reinterpret_cast<uint32_t*>(codes + (lane * I::kPer + h) * 8);
#pragma unroll
      for (int q = 0; q < 4; q++)
        mine[(((wave >> 2) * 4 + q) ^ (lane & 7)) * 4 + (wave & 3)] =
            codes8([&](int j) { return I::value(&w[q * 8 + j], h); }, b);
      if (wave % PER == 0 && c + h < a.cols && r0 < (int)words * 8) {
        const uint64_t o = (g * a.cols + c + h) * (words * 8 / BLOCK) + r0 / BLOCK;
        a.scales[o] = (uint16_t)b.bits;
        if (zeros) a.zeros[o] = (uint8_t)b.zero;
      }
    }
    __syncthreads();
    const uint64_t row0 = g * a.cols + c0;  // of the result
    const uint32_t chunks = words / 4;      // of 16 bytes of a result's row
#pragma unroll
    for (int i = 0; i < C * 8 / 512; i++) {
      const int s = i * 512 + tid, col = s >> 3, k = s & 7;
      if (c0 + col < a.cols && k0 / 32 + k < chunks)
        reinterpret_cast<i32x4*>(a.codes)[(row0 + col) * chunks + k0 / 32 + k] = codes[col * 8 + (k ^ (col / I::kPer & 7))];
    }
    __syncthreads();
  }
}

// The values of a word, (q - z) s.  The difference is exact, and so is its product with a scale
// of 11 bits: the rounding to O is the only one.  (q s - z s is no way to it: with a scale past
// 2^128 / 15 its parts overflow where their difference does not.)
template <typename O>
__device__ __forceinline__ void decode8(uint32_t w, float s, float z, Pack<O, 8>* out) {
  const uint32_t lo = w & kCodeMask, hi = w >> 4 & kCodeMask;
#pragma unroll
  for (int j = 0; j < 8; j++)
    out->v[j] = (O)(((float)((j < 4 ? lo : hi) >> 8 * (j & 3) & 255u) - z) * s);
}

// Rows without padding or gaps, one after another: every chunk of codes lies where its
// values go.  A workgroup takes 1024 consecutive chunks, 4 loads to a lane under way
// (64 x 2048 x 1024 bf16: 57 us, 5.9 TB/s; row by row 104).
template <typename O, int BLOCK>
__global__ __launch_bounds__(256) void gq_dequantize_flat(GqDequantArgs a, uint64_t chunks) {
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.q.codes);
  Pack<O, 8>* out = static_cast<Pack<O, 8>*>(a.out);
  for (uint64_t b = blockIdx.x; b * 1024 < chunks; b += gridDim.x) {
    const uint64_t i = b * 1024 + threadIdx.x, at = b * 1024 + stored(threadIdx.x);
    uint32_t w[4], s[4], z[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      z[j] = 8;
      if (i + j * 256 >= chunks) continue;  // chunks come in sixteens, as the order of words does
      const uint64_t block = (i + j * 256) / (BLOCK / 8);
      w[j] = codes[at + j * 256];
      s[j] = a.q.scales[block];
      if (a.q.zeros) z[j] = a.q.zeros[block];
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (i + j * 256 < chunks) decode8(w[j], scale_of(s[j], a.half), (float)z[j], out + i + j * 256);
  }
}

template <typename O, int BLOCK>
__global__ __launch_bounds__(256) void gq_dequantize(GqDequantArgs a, RowPass pass) {
  const uint64_t step = (uint64_t)gridDim.x * 4 * kRun;
  for (uint64_t s0 = first_segment(); s0 < pass.total; s0 += step) {
#pragma unroll
    for (int i = 0; i < kRun; i++) {
      uint64_t line;
      uint32_t chunk;
      const bool on = pass.locate(s0 + i, &line, &chunk);
      const int left = on ? a.cols - (int)chunk * 8 : 0;
      if (left <= 0) continue;
      const uint32_t w = reinterpret_cast<const uint32_t*>(a.q.codes)[line * pass.chunks + stored(chunk)];
      const uint64_t b = line * (pass.chunks / (BLOCK / 8)) + chunk / (BLOCK / 8);
      const float s = scale_of(a.q.scales[b], a.half), z = a.q.zeros ? (float)a.q.zeros[b] : 8.f;
      const uint64_t g = a.groups == 1 ? 0 : pass.quotient(line, a.rows), r = line - g * a.rows;
      O* p = static_cast<O*>(a.out) + g * a.gso + r * a.ldo + chunk * 8;
      Pack<O, 8> v;
      decode8(w, s, z, &v);
      if (left >= 8) {
        *reinterpret_cast<Pack<O, 8>*>(p) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (j < left) p[j] = v.v[j];
      }
    }
  }
}

template <typename I, int BLOCK>
hipError_t run_quantize(int axis, const GqQuantArgs& a, hipStream_t s) {
  if (axis) {
    // a stack without gaps is one matrix
    GqQuantArgs f = a;
    if (a.gsx == (uint64_t)a.rows * a.ldx && (uint64_t)a.rows * a.groups < (1u << 30)) {
      f.rows = a.rows * a.groups;
      f.groups = 1;
    }
    const RowPass pass(f.groups, f.rows, f.cols);
    gq_quantize_rows<I, BLOCK><<<dim3(row_grid(pass)), dim3(256), 0, s>>>(f, pass);
  } else {
    const uint64_t btiles = ((uint64_t)a.rows + 255) / 256, cols = 64 * I::kPer;
    const dim3 grid(pass_grid(btiles * ((a.cols + cols - 1) / cols) * a.groups, 1 << 20));
    const uint64_t line = 128 / sizeof(typename I::T);  // values
    if (a.cols % line == 0 && a.ldx % line == 0 && a.gsx % line == 0 && reinterpret_cast<uintptr_t>(a.x) % 128 == 0)
      gq_quantize_cols<I, BLOCK, true><<<grid, dim3(512), 0, s>>>(a);
    else
      gq_quantize_cols<I, BLOCK, false><<<grid, dim3(512), 0, s>>>(a);
  }
  return hipGetLastError();
}
template <typename I>
hipError_t quantize_by_block(int axis, int block, const GqQuantArgs& a, hipStream_t s) {
  if (block == 32) return run_quantize<I, 32>(axis, a, s);
  if (block == 64) return run_quantize<I, 64>(axis, a, s);
  return run_quantize<I, 128>(axis, a, s);
}

template <typename O, int BLOCK>
hipError_t run_dequantize(const GqDequantArgs& a, hipStream_t s) {
  if (a.groups == 1 && a.cols % kMxColsPad == 0 && (a.rows == 1 || a.ldo == (uint64_t)a.cols)) {
    const uint64_t chunks = (uint64_t)a.rows * a.cols / 8;
    gq_dequantize_flat<O, BLOCK><<<dim3(pass_grid((chunks + 1023) / 1024, 1 << 20)), dim3(256), 0, s>>>(a, chunks);
  } else {
    const RowPass pass(a.groups, a.rows, a.cols);
    gq_dequantize<O, BLOCK><<<dim3(row_grid(pass)), dim3(256), 0, s>>>(a, pass);
  }
  return hipGetLastError();
}
template <typename O>
hipError_t dequantize_by_block(int block, const GqDequantArgs& a, hipStream_t s) {
  if (block == 32) return run_dequantize<O, 32>(a, s);
  if (block == 64) return run_dequantize<O, 64>(a, s);
  return run_dequantize<O, 128>(a, s);
}

}  // namespace

hipError_t launch_gq_quantize(int dtype, int axis, int block, const GqQuantArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  if (dtype == CIERA_BF16) return quantize_by_block<GqBf16>(axis, block, a, s);
  if (dtype == CIERA_FP16) return quantize_by_block<GqFp16>(axis, block, a, s);
  return quantize_by_block<GqFp32>(axis, block, a, s);
}

hipError_t launch_gq_dequantize(int dtype, int block, const GqDequantArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  GqDequantArgs f = a;
  if (a.gso == (uint64_t)a.rows * a.ldo && (uint64_t)a.rows * a.groups < (1u << 30)) {
    f.rows = a.rows * a.groups;
    f.groups = 1;
  }
  if (dtype == CIERA_BF16) return dequantize_by_block<__bf16>(block, f, s);
  if (dtype == CIERA_FP16) return dequantize_by_block<_Float16>(block, f, s);
  return dequantize_by_block<float>(block, f, s);
}

}  // namespace ciera
