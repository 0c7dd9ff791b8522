// Reductions and scans of 64-bit values over a wave and a workgroup (wave64 DPP and swaps).
#pragma once

#include <stdint.h>

#include "common.h"

namespace q4moe {

__device__ __forceinline__ uint64_t pair64(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }

// op over the values of kLanes neighbouring lanes (16, 32 or the wave), in every lane; both
// partners of a step combine the same two.
template <int kLanes = kWave, typename Op>
__device__ __forceinline__ uint64_t wave_reduce_u64(uint64_t v, Op op) {
  v = op(v, pair64(dpp_u32<kDppQuadXor1>((uint32_t)v), dpp_u32<kDppQuadXor1>((uint32_t)(v >> 32))));
  v = op(v, pair64(dpp_u32<kDppQuadXor2>((uint32_t)v), dpp_u32<kDppQuadXor2>((uint32_t)(v >> 32))));
  v = op(v, pair64(dpp_u32<kDppRowHalfMirror>((uint32_t)v), dpp_u32<kDppRowHalfMirror>((uint32_t)(v >> 32))));
  v = op(v, pair64(dpp_u32<kDppRowMirror>((uint32_t)v), dpp_u32<kDppRowMirror>((uint32_t)(v >> 32))));
  if constexpr (kLanes == 16) return v;
  uint32_t al, bl, ah, bh;
  swap_rows16((uint32_t)v, al, bl);
  swap_rows16((uint32_t)(v >> 32), ah, bh);
  v = op(pair64(al, ah), pair64(bl, bh));
  if constexpr (kLanes == 32) return v;
  swap_halves32((uint32_t)v, al, bl);
  swap_halves32((uint32_t)(v >> 32), ah, bh);
  return op(pair64(al, ah), pair64(bl, bh));
}

template <int kLanes = kWave>
__device__ __forceinline__ double wave_sum_f64(double v) {
  return __longlong_as_double((long long)wave_reduce_u64<kLanes>((uint64_t)__double_as_longlong(v), [](uint64_t a, uint64_t b) {
    return (uint64_t)__double_as_longlong(__longlong_as_double((long long)a) + __longlong_as_double((long long)b));
  }));
}
template <int kLanes = kWave>
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  return wave_reduce_u64<kLanes>(v, [](uint64_t a, uint64_t b) { return max(a, b); });
}
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
  return wave_reduce_u64(v, [](uint64_t a, uint64_t b) { return a + b; });
}

// The sum of the lanes up to and with this one: shifts inside the 16-lane rows, then the rows'
// last lanes to the rows after them.
constexpr int kDppRowShr = 0x110, kDppRowBcast15 = 0x142, kDppRowBcast31 = 0x143;

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {  // 0 where the step brings nothing
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_or_zero(uint64_t v) {
  return pair64(dpp_or_zero<CTRL, ROWS>((uint32_t)v), dpp_or_zero<CTRL, ROWS>((uint32_t)(v >> 32)));
}
template <typename T>
__device__ __forceinline__ T wave_prefix(T v) {
  v += dpp_or_zero<kDppRowShr + 1, 0xF>(v);
  v += dpp_or_zero<kDppRowShr + 2, 0xF>(v);
  v += dpp_or_zero<kDppRowShr + 4, 0xF>(v);
  v += dpp_or_zero<kDppRowShr + 8, 0xF>(v);
  v += dpp_or_zero<kDppRowBcast15, 0xA>(v);
  v += dpp_or_zero<kDppRowBcast31, 0xC>(v);
  return v;
}

}  // namespace q4moe
