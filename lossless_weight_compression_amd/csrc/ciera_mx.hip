// Microscaled 4-bit floating point: quantisation, its reverse, and the product
// of two 4-bit matrices.
//
// A block of 32 values v shares the scale 2^e, e = floor(log2(max |v|)) - 2 (the
// largest of the 4-bit magnitudes 0 .5 1 1.5 2 3 4 6 has exponent 2), kept as the
// byte e + 127 and never below 0; each value is the nearest magnitude to
// |v| 2^-e, ties to the even code, above 6 the 6 itself, with v's sign in bit 3.
#include "ciera.h"
#include "ciera_ops_internal.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

struct Bf16In {
  typedef uint16_t T;
  static __device__ __forceinline__ float f(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
};
struct Fp16In {
  typedef uint16_t T;
  static __device__ __forceinline__ float f(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
};
struct Fp32In {
  typedef float T;
  static __device__ __forceinline__ float f(float v) { return v; }
};

// Scale byte of a block from the bits of its largest magnitude: the exponent
// field less 2.  Integer order of magnitudes puts NaN above infinity above all
// finite values; both give 255, the scale NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255 ? 255u : f > 2 ? f - 2 : 0u;
}
// 2^(byte - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}
// 8 values to 8 codes, the first in the low nibble: the conversion divides by the
// scale, rounds to nearest even and stops at 6.  A block with infinities or NaN
// holds zeros behind its NaN scale.
__device__ __forceinline__ uint32_t encode8(const float* v, uint32_t byte) {
  if (byte == 255) return 0;
  const float s = scale_value(byte);
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
}
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// Blocks along the rows of x: 4 lanes to a block, 8 values each.
template <typename I>
__global__ __launch_bounds__(256) void mx_quantize_rows(MxQuantArgs a) {
  const int kp = (a.cols + (int)kMxColsPad - 1) / (int)kMxColsPad * (int)kMxColsPad;
  const uint64_t chunks = (uint64_t)kp / 8;  // of a row; a multiple of 16
  const uint64_t total = chunks * a.rows * a.groups;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (uint64_t)gridDim.x * 256) {
    const uint64_t line = i / chunks;
    const int c = (int)(i % chunks) * 8;
    const uint64_t g = line / a.rows, r = line % a.rows;
    const typename I::T* p = static_cast<const typename I::T*>(a.x) + g * a.gsx + r * a.ldx + c;
    float v[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      v[j] = c + j < a.cols ? I::f(p[j]) : 0.f;
      m = max(m, magnitude_bits(v[j]));
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const uint32_t byte = scale_byte(m);
    reinterpret_cast<uint32_t*>(a.codes)[i] = encode8(v, byte);
    if ((i & 3) == 0) a.scales[i / 4] = (uint8_t)byte;
  }
}

// Blocks along the columns of x: row c of the result is column c of x.
template <typename I>
__global__ __launch_bounds__(256) void mx_quantize_cols(MxQuantArgs a) {
  const uint64_t blocks = ((uint64_t)a.rows + kMxColsPad - 1) / kMxColsPad * (kMxColsPad / kMxBlock);
  const uint64_t total = blocks * a.cols * a.groups;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (uint64_t)gridDim.x * 256) {
    const int c = (int)(i % a.cols);
    const uint64_t b = i / a.cols % blocks, g = i / a.cols / blocks;
    const typename I::T* p = static_cast<const typename I::T*>(a.x) + g * a.gsx + c;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; j++) {
      const uint64_t r = b * 32 + j;
      v[j] = r < (uint64_t)a.rows ? I::f(p[r * a.ldx]) : 0.f;
      m = max(m, magnitude_bits(v[j]));
    }
    const uint32_t byte = scale_byte(m);
    const uint64_t o = (g * a.cols + c) * blocks + b;
    uint32_t* q = reinterpret_cast<uint32_t*>(a.codes) + o * 4;
#pragma unroll
    for (int j = 0; j < 4; j++) q[j] = encode8(v + 8 * j, byte);
    a.scales[o] = (uint8_t)byte;
  }
}

template <typename O>
__global__ __launch_bounds__(256) void mx_dequantize(MxDequantArgs a) {
  const int kp = (a.cols + (int)kMxColsPad - 1) / (int)kMxColsPad * (int)kMxColsPad;
  const uint64_t chunks = (uint64_t)kp / 8;
  const uint64_t total = chunks * a.rows * a.groups;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (uint64_t)gridDim.x * 256) {
    const uint64_t line = i / chunks;
    const int c = (int)(i % chunks) * 8;
    if (c >= a.cols) continue;
    const uint64_t g = line / a.rows, r = line % a.rows;
    const uint32_t w = reinterpret_cast<const uint32_t*>(a.codes)[i];
    const uint32_t byte = a.scales[i / 4];
    const float s = scale_value(byte), nan = __builtin_nanf("");
    const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
    const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    const float v[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
    O* p = static_cast<O*>(a.out) + g * a.gso + r * a.ldo + c;
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (c + j < a.cols) p[j] = (O)(byte == 255 ? nan : v[j]);
  }
}

// out = a b^T on the rows of every group: the 4-bit matrix instruction takes 128
// contraction steps, a lane's 32 codes and their one scale.
template <typename O, int BM, int BN>
__global__ __launch_bounds__(256) void mx_mm_general(MxMmArgs a) {
  constexpr int CH = 4;  // 16-byte chunks (32 codes) of a row per step of 128
  constexpr int NA = BM * CH / 256, NB = BN * CH / 256, WM = BM / 2 / 16, WN = BN / 2 / 16;
  __shared__ i32x4 la[2][BM * CH];
  __shared__ i32x4 lb[2][BN * CH];
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  const int mleft = t.count - t.m * BM, n0 = tn * BN, nleft = a.n - n0;
  const uint64_t cb = a.kp / 2, sb = a.kp / 32;  // bytes of a row's codes and scales
  const uint8_t* pa = a.a + row * cb;
  const uint8_t* psa = a.sa + row * sb;
  const uint64_t brow = (uint64_t)t.g * a.n + n0;
  const uint8_t* pb = a.b + brow * cb;
  const uint8_t* psb = a.sb + brow * sb;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int r0 = (wave >> 1) * (BM / 2), c0 = (wave & 1) * (BN / 2);
  auto pos = [](int r, int c) { return r * CH + (c ^ ((r >> 2) & 3)); };

  i32x4 ra[NA], rb[NB];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < NA; i++) {
      const int p = i * 256 + tid, r = p / CH, c = p % CH;
      ra[i] = r < mleft ? *reinterpret_cast<const i32x4*>(pa + r * cb + s * 64 + c * 16) : i32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < NB; i++) {
      const int p = i * 256 + tid, r = p / CH, c = p % CH;
      rb[i] = r < nleft ? *reinterpret_cast<const i32x4*>(pb + r * cb + s * 64 + c * 16) : i32x4{0, 0, 0, 0};
    }
  };
  auto put = [&](int s) {
#pragma unroll
    for (int i = 0; i < NA; i++) la[s][pos((i * 256 + tid) / CH, (i * 256 + tid) % CH)] = ra[i];
#pragma unroll
    for (int i = 0; i < NB; i++) lb[s][pos((i * 256 + tid) / CH, (i * 256 + tid) % CH)] = rb[i];
  };
  f32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; i++)
#pragma unroll
    for (int j = 0; j < WN; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  const int steps = a.kp / 128;
  if (steps) {
    load(0);
    put(0);
  }
  __syncthreads();
  for (int s = 0; s < steps; s++) {
    const bool more = s + 1 < steps;
    if (more) load(s + 1);
    const int cur = s & 1;
    i32x8 fa[WM], fb[WN];
    int xa[WM], xb[WN];
#pragma unroll
    for (int i = 0; i < WM; i++) {
      const int r = r0 + i * 16 + (lane & 15);
      const i32x4 v = la[cur][pos(r, lane >> 4)];
      fa[i] = i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      xa[i] = r < mleft ? psa[r * sb + s * 4 + (lane >> 4)] : 0;
    }
#pragma unroll
    for (int j = 0; j < WN; j++) {
      const int r = c0 + j * 16 + (lane & 15);
      const i32x4 v = lb[cur][pos(r, lane >> 4)];
      fb[j] = i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      xb[j] = r < nleft ? psb[r * sb + s * 4 + (lane >> 4)] : 0;
    }
#pragma unroll
    for (int i = 0; i < WM; i++)
#pragma unroll
      for (int j = 0; j < WN; j++)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i], acc[i][j], 4, 4, 0, xb[j], 0, xa[i]);
    if (more) put(cur ^ 1);
    __syncthreads();
  }
  O* out = static_cast<O*>(a.out) + row * a.ldo + n0;
#pragma unroll
  for (int i = 0; i < WM; i++) {
    const int m = r0 + i * 16 + (lane & 15);
    if (m >= mleft) continue;
#pragma unroll
    for (int j = 0; j < WN; j++) store4(out + (uint64_t)m * a.ldo, c0 + j * 16 + (lane >> 4) * 4, nleft, acc[i][j]);
  }
}

// Workgroups of a pass over `work` items of one thread each; beyond the limit
// each takes several in turn.
uint32_t pass_grid(uint64_t work) {
  const uint64_t g = (work + 255) / 256;
  return (uint32_t)(g < 65536 ? g : 65536);
}

template <typename O>
hipError_t run_mx_mm(const MxMmArgs& a, hipStream_t s) {
  constexpr int BM = 128, BN = 128;
  const uint64_t rows = a.rows, groups = a.groups;
  const uint64_t mt = groups == 1 ? (rows + BM - 1) / BM : rows / BM + (groups < rows ? groups : rows);
  const uint64_t grid = (mt * ((a.n + BN - 1) / BN) + kXcds - 1) / kXcds * kXcds;
  if (grid * 256 >> 32) return hipErrorInvalidConfiguration;
  mx_mm_general<O, BM, BN><<<dim3((uint32_t)grid), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(int dtype, int axis, bool flat, const MxQuantArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  const uint64_t kp = ((uint64_t)(axis ? a.cols : a.rows) + kMxColsPad - 1) / kMxColsPad * kMxColsPad;
  if (axis) {
    const dim3 grid(pass_grid(kp / 8 * a.rows * a.groups));
    if (dtype == CIERA_BF16) mx_quantize_rows<Bf16In><<<grid, dim3(256), 0, s>>>(a);
    else if (dtype == CIERA_FP16) mx_quantize_rows<Fp16In><<<grid, dim3(256), 0, s>>>(a);
    else mx_quantize_rows<Fp32In><<<grid, dim3(256), 0, s>>>(a);
  } else {
    const dim3 grid(pass_grid(kp / kMxBlock * a.cols * a.groups));
    if (dtype == CIERA_BF16) mx_quantize_cols<Bf16In><<<grid, dim3(256), 0, s>>>(a);
    else if (dtype == CIERA_FP16) mx_quantize_cols<Fp16In><<<grid, dim3(256), 0, s>>>(a);
    else mx_quantize_cols<Fp32In><<<grid, dim3(256), 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(int dtype, bool flat, const MxDequantArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  const uint64_t kp = ((uint64_t)a.cols + kMxColsPad - 1) / kMxColsPad * kMxColsPad;
  const dim3 grid(pass_grid(kp / 8 * a.rows * a.groups));
  if (dtype == CIERA_BF16) mx_dequantize<__bf16><<<grid, dim3(256), 0, s>>>(a);
  else if (dtype == CIERA_FP16) mx_dequantize<_Float16><<<grid, dim3(256), 0, s>>>(a);
  else mx_dequantize<float><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx_mm(int out_dtype, const MxMmArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  if (out_dtype == CIERA_BF16) return run_mx_mm<__bf16>(a, s);
  if (out_dtype == CIERA_FP16) return run_mx_mm<_Float16>(a, s);
  return run_mx_mm<float>(a, s);
}

}  // namespace ciera
