// Reductions and scans of 64-bit values over a wave and a workgroup (wave64 DPP and swaps).
#pragma once

#include <stdint.h>

#include "common.h"

namespace q4moe {

__device__ __forceinline__ uint64_t pair64(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }

// op over the wave's values, in every lane; both partners of a step combine the same two.
template <typename Op>
__device__ __forceinline__ uint64_t wave_reduce_u64(uint64_t v, Op op) {
  v = op(v, pair64(dpp_u32<kDppQuadXor1>((uint32_t)v), dpp_u32<kDppQuadXor1>((uint32_t)(v >> 32))));
  v = op(v, pair64(dpp_u32<kDppQuadXor2>((uint32_t)v), dpp_u32<kDppQuadXor2>((uint32_t)(v >> 32))));
  v = op(v, pair64(dpp_u32<kDppRowHalfMirror>((uint32_t)v), dpp_u32<kDppRowHalfMirror>((uint32_t)(v >> 32))));
  v = op(v, pair64(dpp_u32<kDppRowMirror>((uint32_t)v), dpp_u32<kDppRowMirror>((uint32_t)(v >> 32))));
  uint32_t al, bl, ah, bh;
  swap_rows16((uint32_t)v, al, bl);
  swap_rows16((uint32_t)(v >> 32), ah, bh);
  v = op(pair64(al, ah), pair64(bl, bh));
  swap_halves32((uint32_t)v, al, bl);
  swap_halves32((uint32_t)(v >> 32), ah, bh);
  return op(pair64(al, ah), pair64(bl, bh));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
  return __longlong_as_double((long long)wave_reduce_u64((uint64_t)__double_as_longlong(v), [](uint64_t a, uint64_t b) {
    return (uint64_t)__double_as_longlong(__longlong_as_double((long long)a) + __longlong_as_double((long long)b));
  }));
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  return wave_reduce_u64(v, [](uint64_t a, uint64_t b) { return max(a, b); });
}
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
  return wave_reduce_u64(v, [](uint64_t a, uint64_t b) { return a + b; });
}

// The sum of the lanes up to and with this one.
template <typename T>
__device__ __forceinline__ T wave_prefix(T v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const T o = __shfl_up(v, d, kWave);
    if (lane_id() >= d) v += o;
  }
  return v;
}

}  // namespace q4moe
