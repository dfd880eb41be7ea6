// 4-bit integers with group scales: words of codes, scales.
//
// A word holds 8 consecutive values, byte b the codes of values b and b + 4.  The nibbles of
// a byte, taken as an 8-bit float (4 exponent, 3 mantissa bits), are its subnormals and first
// binade: q 2^-9 exactly.  So one conversion with the scale 2^9 makes two codes two-byte
// floats, 7 vector instructions to a word (shifting codes into the mantissa of 16 took 8, and
// left 16 + q to be corrected: 41 clocks a word with the matrix instruction, for 47).
#pragma once
#include "ciera_tiles.h"

namespace ciera {
namespace {

// A scale's value: fp16, or bf16 in the lower half of a word.  half: all ones or zero.  (A
// branch on the type would end the counting of loads under way.)
__device__ __forceinline__ float scale_of(uint32_t bits, uint32_t half) {
  const uint32_t h = __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)bits));
  return __builtin_bit_cast(float, (h & half) | (bits << 16 & ~half));
}

// 8 codes as two-byte floats, in order.
constexpr uint32_t kCodeMask = 0x0f0f0f0fu;
__device__ __forceinline__ bf16x8 expand(uint32_t w, Bf16) {
  const uint32_t lo = w & kCodeMask, hi = w >> 4 & kCodeMask;
  return __builtin_bit_cast(
      bf16x8, i32x4{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false)),
                    __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true)),
                    __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false)),
                    __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true))});
}
__device__ __forceinline__ f16x8 expand(uint32_t w, Fp16) {
  const uint32_t lo = w & kCodeMask, hi = w >> 4 & kCodeMask;
  return __builtin_bit_cast(
      f16x8, i32x4{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, false)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, true)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, false)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, true))});
}
__device__ __forceinline__ bf16x8 ones(Bf16) {
  return __builtin_bit_cast(bf16x8, i32x4{0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80});
}
__device__ __forceinline__ f16x8 ones(Fp16) {
  return __builtin_bit_cast(f16x8, i32x4{0x3c003c00, 0x3c003c00, 0x3c003c00, 0x3c003c00});
}

}  // namespace
}  // namespace ciera
