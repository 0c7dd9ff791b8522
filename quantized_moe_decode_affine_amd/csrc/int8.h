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

// Eight consecutive values of a row as they lie in memory.
template <typename In>
struct I8Chunk {
  typedef In vec_t __attribute__((ext_vector_type(8)));
  vec_t raw;
  __device__ __forceinline__ void load(const In* p) { raw = *reinterpret_cast<const vec_t*>(p); }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (sizeof(In) == 2) return bf16_bits_to_f32(raw[j]);
    else return raw[j];
  }
  // Bits of the largest magnitude among them and `m`.
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(at(j)) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint2 codes(const I8Rounder& rd) const {
    return make_uint2(rd.pack4(at(0), at(1), at(2), at(3)), rd.pack4(at(4), at(5), at(6), at(7)));
  }
};

// A row of K values to its codes and scale, by one wave.  Up to kHeld chunks of 8 values per
// lane stay in registers between the largest magnitude and the codes, the rest of a longer
// row is read again (from the caches).
template <int kHeld, typename In>
__device__ __forceinline__ void i8_quantize_row(const In* x, int K, int8_t* codes, float* scale_out) {
  const int lane = lane_id();
  I8Chunk<In> held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i].load(x + min((i * kWave + lane) * 8, K - 8));
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) most = held[i].most(most);
  for (int j = (kHeld * kWave + lane) * 8; j < K; j += kWave * 8) {
    I8Chunk<In> v;
    v.load(x + j);
    most = v.most(most);
  }
  const float scale = i8_scale(wave_max_u32(most));
  const I8Rounder rd(scale);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = (i * kWave + lane) * 8;
    if (j < K) *reinterpret_cast<uint2*>(codes + j) = held[i].codes(rd);
  }
  for (int j = (kHeld * kWave + lane) * 8; j < K; j += kWave * 8) {
    I8Chunk<In> v;
    v.load(x + j);
    *reinterpret_cast<uint2*>(codes + j) = v.codes(rd);
  }
  if (lane == 0) *scale_out = scale;
}

// fp32 -> bf16 bits, nearest even; a NaN stays a NaN (the bare carry could turn it into 0 or infinity).
__device__ __forceinline__ uint16_t i8_bf16(float f) {
  return (uint16_t)(f == f ? f32_to_bf16_bits(f) : 0x7FC0u);
}

// The experts' arithmetic on exact integer sums, one rounding an operation and in this order
// wherever it is done (a fused multiply-add in one kernel and not in another would move the
// last bit): a token gets the same bits whichever kernels its batch takes.
__device__ __forceinline__ float i8_scaled(float sum, float row_scale, float channel_scale) {
#pragma clang fp contract(off)
  return sum * row_scale * channel_scale;
}
__device__ __forceinline__ float i8_swiglu(float g, float u) {
#pragma clang fp contract(off)
  return g / (1.0f + expf(-g)) * u;
}
__device__ __forceinline__ float i8_add_slot(float y, float out, float weight) {
#pragma clang fp contract(off)
  return y + out * weight;
}

}  // namespace q4moe
