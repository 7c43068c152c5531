// Values held in 8 bits: e4m3 codes with one power of two for a head's values,
// kept as the byte that is its exponent in fp32 (gfx950).
//
// The scale is a power of two so that no reader rounds again: a code times its
// scale is a number of the row's 16-bit type.  e4m3 is itself a floating type,
// so a scale places its 18 binades and adds nothing to the values' precision: a
// scale for a head's values, not for every 128 of them, loses only what lies
// 2^-14 below the head's largest value.
#pragma once

#include "row_format.h"

namespace gpb {

// Range of a scale's exponent and the largest value held, by the row's type: a
// code's smallest step, 2^-9 scales, is a number of the type (fp16: its smallest,
// 2^-24), and so is the largest code that a scale of 2^kMost takes, 240.
template <typename T>
struct Held;
template <>
struct Held<__bf16> {
  static constexpr int kLeast = -100, kMost = 120;
  static constexpr float kTop = 0x1.ep127f;
};
template <>
struct Held<_Float16> {
  static constexpr int kLeast = -15, kMost = 8;
  static constexpr float kTop = 0x1.ep15f;
};

// x within what is held; NaN stays.
template <typename T>
__device__ __forceinline__ float within(float x) {
  return x != x ? x : __builtin_fminf(__builtin_fmaxf(x, -Held<T>::kTop), Held<T>::kTop);
}

// The exponent of the scale of values of which the largest is `top` (>= 0, held).
// top = 1.f 2^(n - 127) is at most 448 2^e = 1.75 2^(8 + e): e is n - 135, one more
// where f is beyond 0.75.  Zeros and subnormals come out below every kLeast.
template <typename T>
__device__ __forceinline__ int scale_exponent(float top) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, top);
  const int e = static_cast<int>(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u);
  return e < Held<T>::kLeast ? Held<T>::kLeast : e > Held<T>::kMost ? Held<T>::kMost : e;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(e + 127) << 23);
}

// Codes of four values, x = value / scale (|x| <= 448).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// The scale of a scale byte.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __builtin_bit_cast(float, byte << 23);
}

// What eight codes stand for.  Exact: the type has the codes' four bits, and every
// exponent that an append's scale gives them.
template <typename T>
__device__ __forceinline__ typename Vec<T>::x8 values8(u32x2 codes, float scale) {
  typename Vec<T>::x8 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t four = codes[i / 2];
    if constexpr (__is_same(T, _Float16)) {
      const auto two = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(four, scale, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(four, scale, false);
      x[2 * i] = two[0];
      x[2 * i + 1] = two[1];
    } else {
      const auto two = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, scale, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, scale, false);
      x[2 * i] = two[0];
      x[2 * i + 1] = two[1];
    }
  }
  return x;
}

}  // namespace gpb
