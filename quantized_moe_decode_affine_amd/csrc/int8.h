// Symmetric 8-bit rows: codes q in -127..127 and one fp32 scale per row, x ~ scale * q.
//   scale = fl32(max|x| / 127)   q = x / scale rounded to the nearest integer, ties to even
// A row of zeros (or one whose scale underflows to 0) has scale 0 and codes 0; a row that
// holds an infinity or a NaN has scale NaN and codes 0, so whatever is computed from it is NaN.
#pragma once

#include <stdint.h>

#include "common.h"

namespace q4moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// The scale of a row whose largest magnitude has the bits `most` (sign clear; a NaN's bits
// lie above infinity's, so an integer maximum keeps it).
__device__ __forceinline__ float i8_scale(uint32_t most) {
  return most < 0x7F800000u ? __uint_as_float(most) / 127.0f : __uint_as_float(0x7FC00000u);
}

// Rounds a row's values to codes.  The quotient is taken as x * (1/scale), which is off by
// less than half a step and can only miss the nearest integer next to a border, where the
// remainder x - q*scale decides: it is exact in fp32 (a multiple of scale's last bit, and
// at most scale), so the code is the correctly rounded one.  Scales so small that 1/scale
// would overflow are moved up by a power of two together with x.
struct I8Rounder {
  float mul, s, inv;
  __device__ __forceinline__ explicit I8Rounder(float scale) {
    mul = scale < 0x1p-100f ? 0x1p100f : 1.0f;
    s = scale * mul;
    inv = s > 0.0f ? 1.0f / s : 0.0f;  // zero and NaN scales: codes 0
  }
  __device__ __forceinline__ int operator()(float x) const {
    if (!(s > 0.0f)) return 0;
    const float v = x * mul;
    float q = rintf(v * inv);
    const float r2 = 2.0f * fmaf(-q, s, v);  // twice the remainder: compared with the step itself
    const bool odd = (int)q & 1;
    if (r2 > s || (r2 == s && odd)) q += 1.0f;
    if (r2 < -s || (r2 == -s && odd)) q -= 1.0f;
    return max(-127, min(127, (int)q));
  }
  __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) const {
    return ((uint32_t)(*this)(a) & 0xFFu) | (((uint32_t)(*this)(b) & 0xFFu) << 8) |
           (((uint32_t)(*this)(c) & 0xFFu) << 16) | ((uint32_t)(*this)(d) << 24);
  }
};

// Eight consecutive values of a row as fp32.
__device__ __forceinline__ void i8_load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void i8_load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Bits of the largest magnitude among eight values, and the running maximum before them.
__device__ __forceinline__ uint32_t i8_most(const float (&v)[8], uint32_t most) {
#pragma unroll
  for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return most;
}

}  // namespace q4moe
