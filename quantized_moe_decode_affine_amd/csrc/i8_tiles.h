// The dense 8-bit product's tile by its size: host code alone, no HIP.
#pragma once

#include <stdint.h>

namespace q4moe {

constexpr int kXcds = 8;                       // the grid of dense tiles is a multiple of them
constexpr int64_t kMaxThreads = 0xFFFFFFFFll;  // of a grid

// Rows and columns of a tile (256, 128 or 64) for m rows on n channels, by the time that its
// rounds of workgroups take, in microseconds per 128 columns of K (measured on 8192 x 8192 x
// 4096): 256 x 256, one workgroup on a compute unit, 1.95; 128 x 128, two, 1.14; 64 x 64,
// three, 0.63.  The large tile moves the fewest bytes (that product takes 250, 292 and 430 us),
// a small one spreads few rows over the chip: 512 rows on 2048 x 2048 take 32, 21 and 13 us
// with it.
inline int i8_dense_tile(int64_t m, int64_t n, int64_t cus) {
  auto rounds = [&](int64_t t, int64_t at_once) {
    const int64_t blocks = (m + t - 1) / t * ((n + t - 1) / t);
    if (t < 256 && (blocks + kXcds) * 256 > kMaxThreads) return 1e30;  // more than a grid holds
    return (double)((blocks + cus * at_once - 1) / (cus * at_once));
  };
  const double large = rounds(256, 1) * 1.95, middle = rounds(128, 2) * 1.14, small = rounds(64, 3) * 0.63;
  return large <= middle && large <= small ? 256 : middle <= small ? 128 : 64;
}

}  // namespace q4moe
