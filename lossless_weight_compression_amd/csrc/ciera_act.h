// The gated block's activations and their derivatives, in fp32, and what becomes of the
// products' results.
#pragma once
#include "ciera.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// Both activations are v s(z(v)) with the logistic s(z) = 1 / (1 + exp(-z)): z = v, or
// 2 c (v + 0.044715 v^3), which is the tanh form of GELU: (1 + tanh(y)) / 2 = s(2 y).  So
// far negative v lose no digits to the difference 1 + tanh.  What is left is the rounding of
// exp2's argument, some 2^-23 |z| of the result (3e-6 at z = -60, where the result is 1e-25), and z's
// own in GELU, as large.  Where s would be below 2^-126 it may be 0.
constexpr float kGelu = 1.5957691216057308f, kGeluCube = 0.044715f;  // 2 sqrt(2 / pi)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float act_arg(float v, int act) {
  return act == CIERA_ACT_SILU ? v : kGelu * v * __builtin_fmaf(kGeluCube * v, v, 1.f);
}
// v s, where v may be -infinity and s its 0: the limit is 0.  As unsigned numbers only negative
// NaN lie above -infinity, and a NaN's s is a NaN too: one minimum makes it the lowest number.
__device__ __forceinline__ float times_logistic(float v, float s) {
  return __builtin_bit_cast(float, min(__builtin_bit_cast(uint32_t, v), 0xff7fffffu)) * s;
}
// act(v).  exp(-z) overflows to infinity for far negative z, whose reciprocal is 0.
__device__ __forceinline__ float act_value(float v, int act) {
  return times_logistic(v, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * act_arg(v, act))));
}
// act(v) and act'(v) = s + v s (1 - s) z'(v).  With e = exp(-|z|) <= 1 both s and 1 - s are
// quotients of e and 1 + e: neither is the difference of near numbers.  Where s (1 - s) is
// 0 the second term is, also at infinity, and at -infinity, what a kept G below the range of its
// type becomes, both are 0.
__device__ __forceinline__ void act_grad(float v, int act, float* value, float* slope) {
  const float z = act_arg(v, act), e = __builtin_amdgcn_exp2f(-kLog2e * __builtin_fabsf(z));
  const float r = __builtin_amdgcn_rcpf(1.f + e), s = z < 0.f ? e * r : r, t = e * r * r;
  const float dz = act == CIERA_ACT_SILU ? 1.f : kGelu * __builtin_fmaf(3.f * kGeluCube * v, v, 1.f);
  *value = times_logistic(v, s);
  *slope = t > 0.f ? __builtin_fmaf(v * t, dz, s) : s;
}

// a b rounded to 32 bits by itself.  The compiler makes some of the products that are then rounded
// to fp16 one instruction with one rounding, others two: the last bit of an element would go by
// where in which kernel it is computed, so that h would differ with G and U kept or not.
__device__ __forceinline__ float product(float a, float b) {
  float v = a * b;
  asm("" : "+v"(v));
  return v;
}

// act(G) U of 4 columns.
__device__ __forceinline__ f32x4 gated(f32x4 g, f32x4 u, int act) {
  f32x4 h;
#pragma unroll
  for (int i = 0; i < 4; i++) h[i] = product(act_value(g[i], act), u[i]);
  return h;
}

// Where a tile of the gated block goes: h, and G and U where they are kept.
template <typename O>
struct GluOut {
  typedef O T;
  O *out, *gate, *up;
  uint64_t ldo, ldog, ldou;
  int act;
  __device__ __forceinline__ GluOut at(uint64_t row, int col) const {
    return GluOut{out + row * ldo + col, gate ? gate + row * ldog + col : nullptr, up ? up + row * ldou + col : nullptr,
                  ldo, ldog, ldou, act};
  }
  __device__ __forceinline__ void put(int r, int c, int left, f32x4 glo, f32x4 ghi, f32x4 ulo, f32x4 uhi) const {
    store_row8(out + (uint64_t)r * ldo + c, left, gated(glo, ulo, act), gated(ghi, uhi, act));
    if (gate) {
      store_row8(gate + (uint64_t)r * ldog + c, left, glo, ghi);
      store_row8(up + (uint64_t)r * ldou + c, left, ulo, uhi);
    }
  }
  // of 4 columns; `cols` columns are left from column 0
  __device__ __forceinline__ void put4(int r, int c, int cols, f32x4 g, f32x4 u) const {
    store4(out + (uint64_t)r * ldo, c, cols, gated(g, u, act));
    if (gate) {
      store4(gate + (uint64_t)r * ldog, c, cols, g);
      store4(up + (uint64_t)r * ldou, c, cols, u);
    }
  }
};

// dG = D U act'(G) and dU = D act(G), G and U from memory.  U act'(G) first: D U can be past the
// range where the result is not, and act' is 1.13 at most.
template <typename O>
struct GradOut {
  typedef O T;
  const O *gate, *up;
  O *dgate, *dup;
  uint64_t ldg, ldu, lddg, lddu;
  int act;
  __device__ __forceinline__ GradOut at(uint64_t row, int col) const {
    return GradOut{gate + row * ldg + col, up + row * ldu + col, dgate + row * lddg + col, dup + row * lddu + col,
                   ldg, ldu, lddg, lddu, act};
  }
  __device__ __forceinline__ void put(int r, int c, int left, f32x4 lo, f32x4 hi) const {
    float g[8], u[8];
    load_row8(gate + (uint64_t)r * ldg + c, left, g);
    load_row8(up + (uint64_t)r * ldu + c, left, u);
    f32x4 dg[2], du[2];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float d = i < 4 ? lo[i & 3] : hi[i & 3];
      float value, slope;
      act_grad(g[i], act, &value, &slope);
      dg[i >> 2][i & 3] = product(d, u[i] * slope);
      du[i >> 2][i & 3] = product(d, value);
    }
    store_row8(dgate + (uint64_t)r * lddg + c, left, dg[0], dg[1]);
    store_row8(dup + (uint64_t)r * lddu + c, left, du[0], du[1]);
  }
};

}  // namespace
}  // namespace ciera
