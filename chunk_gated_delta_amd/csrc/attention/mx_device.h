// Rows in codes of 4 or 8 bits with one power-of-two scale for 32 values (a block): sign and magnitude
// on the grid 0 .5 1 1.5 2 3 4 6 (4 bits, the code of an even element in the low half of its byte), or
// sign, four exponent and three mantissa bits up to 448 (8 bits).  Scale byte s stands for 2^(s - 127),
// 255 for not a number.
//
// gfx950 converts two values an instruction in either direction, scale included.  Read with a scale that
// write_block chooses (12 or more), every value is a bf16 without rounding: at most four significant
// bits, and 2^-124 or more in size.  Both directions were compared with the definition over all codes and
// scales, and over all bf16 values, random bit patterns and ties.
#pragma once
#include "attn_device.h"

namespace carve {

typedef unsigned u32;
typedef u32 u32x2 __attribute__((ext_vector_type(2)));
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block from the bits of its largest size.  A value between the last code and half
// a step behind it is held as the last code, so the exponent grows where the mantissa is past 1.75 (4 bits:
// 7 / 4) or 1.8125 (8 bits: 464 / 256).  Not below 12: smaller values of a bf16 or float block are then
// subnormal only where they round to zero, and read values never are.
template <int BITS>
__device__ __forceinline__ u32 mx_scale(u32 big) {
  constexpr u32 carry = BITS == 4 ? 0x1fffffu : 0x17ffffu;
  constexpr int lead = BITS == 4 ? 2 : 8, most = 254 - lead;
  const int e = (int)((big + carry) >> 23) - lead;
  return big >= 0x7f800000u ? 255u : (u32)min(max(e, 12), most);
}
__device__ __forceinline__ float scale_value(u32 s) { return __builtin_bit_cast(float, s << 23); }

// the largest size of the 32 values that four neighbouring lanes hold, as bits
__device__ __forceinline__ u32 quad_max(u32 x) {
  x = max(x, (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0xb1, 0xf, 0xf, false));    // lanes 1 0 3 2
  return max(x, (u32)__builtin_amdgcn_update_dpp(0, (int)x, 0x4e, 0xf, 0xf, false));   // lanes 2 3 0 1
}
__device__ __forceinline__ u32 size_bits(float x) { return __builtin_bit_cast(u32, x) & 0x7fffffffu; }

__device__ __forceinline__ void to_floats(const Frag<bf16>& f, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (float)f.v[j];
}
__device__ __forceinline__ void to_floats(const Frag<float>& f, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = f.lo[j];
    x[4 + j] = f.hi[j];
  }
}

// Eight values of a lane, a quarter of a block that lanes 4 n .. 4 n + 3 hold: its codes, and the
// block's scale byte in every lane of the four.
template <int BITS> struct Eight;
template <> struct Eight<4> { u32 w; };
template <> struct Eight<8> { u32x2 w; };
template <int BITS, typename T>
__device__ __forceinline__ Eight<BITS> write_block(const Frag<T>& f, u32& scale) {
  float x[8];
  to_floats(f, x);
  u32 big = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) big = max(big, size_bits(x[j]));
  scale = mx_scale<BITS>(quad_max(big));
  const float s = scale_value(scale);
  Eight<BITS> c;
  if constexpr (BITS == 4) {
    c.w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], s, 0);
    c.w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.w, x[2], x[3], s, 1);
    c.w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.w, x[4], x[5], s, 2);
    c.w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.w, x[6], x[7], s, 3);
    if (scale == 255u) c.w = 0;
  } else {
    // (the conversion to 8 bits does not stop at the last code by itself)
    const float top = __builtin_bit_cast(float, ((scale + 8) << 23) | 0x600000u);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_fmed3f(x[j], -top, top);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i16x2 w = {0, 0};
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[4 * h], x[4 * h + 1], s, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[4 * h + 2], x[4 * h + 3], s, true);
      c.w[h] = scale == 255u ? 0u : __builtin_bit_cast(u32, w);
    }
  }
  return c;
}

// Two neighbouring values of a word of codes as bf16 (X: which two; 4 bits: 0 .. 3, 8 bits: 0, 1).
template <int BITS, int X>
__device__ __forceinline__ u32 read_pair(u32 w, float s) {
  if constexpr (BITS == 4) return __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, X));
  else return __builtin_bit_cast(u32, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, X != 0));
}
template <int BITS>
__device__ __forceinline__ Frag<bf16> read_eight(const Eight<BITS>& c, float s) {
  u32x4 r;
  if constexpr (BITS == 4)
    r = u32x4{read_pair<4, 0>(c.w, s), read_pair<4, 1>(c.w, s), read_pair<4, 2>(c.w, s), read_pair<4, 3>(c.w, s)};
  else
    r = u32x4{read_pair<8, 0>(c.w[0], s), read_pair<8, 1>(c.w[0], s), read_pair<8, 0>(c.w[1], s), read_pair<8, 1>(c.w[1], s)};
  Frag<bf16> f;
  f.v = __builtin_bit_cast(bf16x8, r);
  return f;
}

}  // namespace carve
