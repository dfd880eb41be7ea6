// 4-bit integer weights with group scales: quantisation and its reverse.
//
// A block of 32, 64 or 128 values v of a row shares a scale s and a zero z (0 to 15, 8 where
// none are kept): code q stands for s (q - z).  With zeros s spreads the 16 codes over the
// block's range, 0 in it: s = (hi - lo) / 15, z = rint(-lo / s), q = rint(v / s) + z, all
// clamped to 0 ... 15; without, s = max |v| / 7.
#include "ciera.h"
#include "ciera_gq.h"
#include "ciera_ops_internal.h"
#include "ciera_rows.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// s rounded to the scales' type, its bits; a scale below 2^-126 becomes 0.
__device__ __forceinline__ uint32_t scale_bits(float s, int half) {
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
  float s, r, z;
  bool bad;
  // of a block with the smallest and the largest value, or (symmetric) the largest magnitude
  // in hi; not finite where one of its values is not
  __device__ __forceinline__ BlockScale(float lo, float hi, bool zeros, int half) {
    const float range = zeros ? (hi - lo) / 15.f : hi / 7.f;
    bits = scale_bits(range, half);
    s = scale_of(bits, half);
    bad = !(s < __builtin_inff());
    if (bad) {
      bits = half ? 0x7e00u : 0x7fc0u;
      s = 0.f;
    }
    r = s > 0.f ? 1.f / s : 0.f;
    z = zeros ? fminf(fmaxf(__builtin_rintf(quotient(-lo, s, r)), 0.f), 15.f) : bad ? 0.f : 8.f;
    zero = (uint32_t)z;
  }
  __device__ __forceinline__ uint32_t code(float v) const {
    return (uint32_t)fminf(fmaxf(__builtin_rintf(quotient(v, s, r)) + z, 0.f), 15.f);
  }
};

// An input type: values from words of memory.
struct GqBf16 {
  typedef uint16_t T;
  static constexpr int kPer = 2;
  static __device__ __forceinline__ float value(const uint32_t* w, int j) {
    return __builtin_bit_cast(float, j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};
struct GqFp16 {
  typedef uint16_t T;
  static constexpr int kPer = 2;
  static __device__ __forceinline__ float value(const uint32_t* w, int j) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(w[j / 2] >> (j & 1 ? 16 : 0)));
  }
};
struct GqFp32 {
  typedef uint32_t T;
  static constexpr int kPer = 1;
  static __device__ __forceinline__ float value(const uint32_t* w, int j) { return __builtin_bit_cast(float, w[j]); }
};

// Smallest and largest of a block.  A value that is not finite must not get lost in the
// comparisons: hi becomes infinite with it.
struct Extent {
  float lo = 0.f, hi = 0.f;
  __device__ __forceinline__ void add(float v, bool zeros) {
    if (zeros) {
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    } else {
      hi = fmaxf(hi, __builtin_fabsf(v));
    }
    if (!(__builtin_fabsf(v) < __builtin_inff())) hi = __builtin_inff();
  }
  __device__ __forceinline__ void join(float l, float h) {
    lo = fminf(lo, l);
    hi = fmaxf(hi, h);
  }
  template <int CTRL>
  __device__ __forceinline__ void across() {  // lanes
    const float l = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, lo), CTRL, 0xf, 0xf, false));
    const float h = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, hi), CTRL, 0xf, 0xf, false));
    join(l, h);
  }
};

// 8 values to a word of codes.
template <typename I>
__device__ __forceinline__ uint32_t codes8(const uint32_t* w, const BlockScale& b) {
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) c |= b.code(I::value(w, j)) << (8 * (j & 3) + (j & 4));
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
      Extent e;
#pragma unroll
      for (int j = 0; j < 8; j++) e.add(I::value(w[i], j), zeros);
      e.across<0xb1>();                       // lane ^ 1
      e.across<0x4e>();                       // lane ^ 2
      if (BLOCK >= 64) e.across<0x141>();     // 7 - lane of 8
      if (BLOCK >= 128) e.across<0x140>();    // 15 - lane of 16
      if (!on[i]) continue;
      const BlockScale b(e.lo, e.hi, zeros, a.half);
      reinterpret_cast<uint32_t*>(a.codes)[line[i] * pass.chunks + stored(chunk[i])] = codes8<I>(w[i], b);
      if (chunk[i] % (BLOCK / 8) == 0) {
        const uint64_t o = line[i] * (pass.chunks / (BLOCK / 8)) + chunk[i] / (BLOCK / 8);
        a.scales[o] = (uint16_t)b.bits;
        if (zeros) a.zeros[o] = (uint8_t)b.zero;
      }
    }
  }
}

// Blocks down the columns of x: row c of the result is column c of x.  A workgroup takes 256
// rows of x, 32 to a wave, of 64 words' columns; a lane holds the 32 values of its one or two
// columns, the waves of one block exchange their extents, and the codes go through LDS.
template <typename I, int BLOCK>
__global__ __launch_bounds__(512) void gq_quantize_cols(GqQuantArgs a) {
  constexpr int C = 64 * I::kPer, PER = BLOCK / 32;  // columns; waves to a block
  __shared__ i32x4 codes[8 * C];
  __shared__ float2 extents[BLOCK > 32 ? 8 : 1][BLOCK > 32 ? C : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool zeros = a.zeros != nullptr;
  const uint32_t words = (uint32_t)((a.rows + (int)kMxColsPad - 1) / (int)kMxColsPad) * (kMxColsPad / 8);  // of a result's row
  const uint32_t btiles = (words + 31) / 32, ctiles = (a.cols + C - 1) / C;
  const uint64_t all = (uint64_t)btiles * ctiles * a.groups;
  for (uint64_t t = blockIdx.x; t < all; t += gridDim.x) {
    const uint64_t g = t / ((uint64_t)btiles * ctiles);
    const uint32_t k0 = (uint32_t)(t / ctiles % btiles) * 256;
    const int c0 = (int)(t % ctiles) * C, c = c0 + lane * I::kPer, r0 = (int)k0 + wave * 32;
    const typename I::T* p = static_cast<const typename I::T*>(a.x) + g * a.gsx + (uint64_t)r0 * a.ldx + c;
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; j++) {
      w[j] = 0;
      if (r0 + j < a.rows && c < a.cols) {
        const typename I::T* at = p + (uint64_t)j * a.ldx;
        w[j] = *at;
        if (I::kPer == 2 && c + 1 < a.cols) w[j] |= (uint32_t)at[1] << 16;
      }
    }
    Extent e[I::kPer];
#pragma unroll
    for (int j = 0; j < 32; j++)
#pragma unroll
      for (int h = 0; h < I::kPer; h++) e[h].add(I::value(&w[j], h), zeros);
    if constexpr (BLOCK > 32) {
#pragma unroll
      for (int h = 0; h < I::kPer; h++) extents[wave][lane * I::kPer + h] = make_float2(e[h].lo, e[h].hi);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < PER; v++)
#pragma unroll
        for (int h = 0; h < I::kPer; h++) {
          const float2 o = extents[wave / PER * PER + v][lane * I::kPer + h];
          e[h].join(o.x, o.y);
        }
    }
#pragma unroll
    for (int h = 0; h < I::kPer; h++) {
      const BlockScale b(e[h].lo, e[h].hi, zeros, a.half);
      const int col = lane * I::kPer + h;
      uint32_t* mine = reinterpret_cast<uint32_t*>(codes + col * 8);
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) v |= b.code(I::value(&w[q * 8 + j], h)) << (8 * (j & 3) + (j & 4));
        mine[(((wave >> 2) * 4 + q) ^ (lane & 7)) * 4 + (wave & 3)] = b.bad ? 0 : v;
      }
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
      f32x4 v[2];
#pragma unroll
      for (int j = 0; j < 8; j++) v[j >> 2][j & 3] = s * ((float)(w >> (8 * (j & 3) + (j & 4)) & 15u) - z);
      store_row8(static_cast<O*>(a.out) + g * a.gso + r * a.ldo + chunk * 8, left, v[0], v[1]);
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
    gq_quantize_cols<I, BLOCK><<<grid, dim3(512), 0, s>>>(a);
  }
  return hipGetLastError();
}
template <typename I>
hipError_t quantize_by_block(int axis, int block, const GqQuantArgs& a, hipStream_t s) {
  if (block == 32) return run_quantize<I, 32>(axis, a, s);
  if (block == 64) return run_quantize<I, 64>(axis, a, s);
  return run_quantize<I, 128>(axis, a, s);
}

template <typename O>
hipError_t dequantize_by_block(int block, const GqDequantArgs& a, const RowPass& pass, hipStream_t s) {
  const dim3 grid(row_grid(pass));
  if (block == 32) gq_dequantize<O, 32><<<grid, dim3(256), 0, s>>>(a, pass);
  else if (block == 64) gq_dequantize<O, 64><<<grid, dim3(256), 0, s>>>(a, pass);
  else gq_dequantize<O, 128><<<grid, dim3(256), 0, s>>>(a, pass);
  return hipGetLastError();
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
  const RowPass pass(f.groups, f.rows, f.cols);
  if (dtype == CIERA_BF16) return dequantize_by_block<__bf16>(block, f, pass, s);
  if (dtype == CIERA_FP16) return dequantize_by_block<_Float16>(block, f, pass, s);
  return dequantize_by_block<float>(block, f, pass, s);
}

}  // namespace ciera
