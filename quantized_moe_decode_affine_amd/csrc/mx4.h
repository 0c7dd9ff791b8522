// Microscaled 4-bit rows: blocks of 32 consecutive columns share a scale, a power of two held
// as its biased exponent (E8M0: 2^(byte - 127), 255 a NaN); an element is e2m1, a sign and one
// of 0, 0.5, 1, 1.5, 2, 3, 4, 6.
//   scale = 2^(floor(log2 max|x|) - 2), at least 2^-127   code = x / scale to the nearest, ties
//   to the even code, beyond 6 to 6
// A block of zeros has scale 2^-127; a block that holds an infinity or a NaN has scale byte 255
// and codes 0, so whatever is computed from it is NaN.
#pragma once

#include <stdint.h>

#include "common.h"
#include "int8.h"

namespace q4moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;

// The scale byte of a block whose largest magnitude has the fp32 bits `most` (sign clear; a
// NaN's bits lie above infinity's).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t most) {
  const uint32_t e = most >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// The scale as a float (255: any finite one, its codes are zeroed).
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x3F800000u : byte << 23);
}

// Eight values to eight codes, the first in the lowest bits.  The conversion divides by the
// scale and rounds to nearest even, values beyond 6 to 6 (checked for every bf16 value).
__device__ __forceinline__ uint32_t mx4_codes(const I8Chunk<uint16_t>& v, uint32_t byte) {
  const float s = mx4_scale(byte);
  const uint4 u = __builtin_bit_cast(uint4, v.raw);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, u.x), s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, u.y), s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, u.z), s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, u.w), s, 3);
  return byte == 255u ? 0u : c;
}
__device__ __forceinline__ uint32_t mx4_codes(const I8Chunk<float>& v, uint32_t byte) {
  const float s = mx4_scale(byte);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.raw[0], v.raw[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.raw[2], v.raw[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.raw[4], v.raw[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v.raw[6], v.raw[7], s, 3);
  return byte == 255u ? 0u : c;
}

// Half a block, 16 values as they lie in memory, to its codes; the lane next to this one (the
// other of an even and an odd one) has the other half.
template <typename In>
struct Mx4Half {
  I8Chunk<In> a, b;
  __device__ __forceinline__ void load(const In* p) {
    a.load(p);
    b.load(p + 8);
  }
  __device__ __forceinline__ uint2 codes(uint32_t* byte) const {
    uint32_t most = b.most(a.most(0u));
    most = max(most, dpp_u32<kDppQuadXor1>(most));
    *byte = mx4_scale_byte(most);
    return make_uint2(mx4_codes(a, *byte), mx4_codes(b, *byte));
  }
};

// Operands of the 4-bit matrix instructions: 32 codes of a row in the low four registers.
__device__ __forceinline__ i32x8_t mx4_operand(i32x4_t v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
constexpr int kFp4 = 4;  // the operands' format in the f8f6f4 instructions

}  // namespace q4moe
