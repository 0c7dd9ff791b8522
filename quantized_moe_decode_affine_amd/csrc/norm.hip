// Root-mean-square norm of rows, with the residual's addition before it and a bf16 or an
// 8-bit result (rms_norm).
//
//   t = bf16(x + r)   y = t / sqrt(sum t^2 / k + eps) * w
//
// One pass: a row's t stay in registers between its sums and its results.  The sum of squares
// and what the codes' borders hang on (y, the largest |t w|, y / scale) are in fp64, so a
// code is the definition's: in fp32 about one code in 50,000 fell on the other side of a
// border.
//
// A bf16 result is bound by memory: 8191 rows of 4096 with a residual take 50 us, 5.4 TB/s (a
// copy of 1 GiB reaches 5.2), 42 us where the last cache holds a part.  Codes on many rows are
// bound by fp64, some ten operations and conversions an element: 4096 rows of 2048 with a residual
// 17.2 us for 59 MB, 3.4 TB/s, where a bf16 result takes 12.9 us for 67 MB.  One row of 2048 takes
// 3 us either way: the launch, a turn of memory and the reduction.
#include <algorithm>

#include "int8.h"
#include "steps.h"
#include "wave64.h"

namespace q4moe {

namespace {

typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));

struct NormArgs {
  const uint16_t *x, *r, *w;  // r: null, or the residual
  int64_t rows;
  int k;
  double eps;
  uint16_t* total;  // with r: bf16(x + r), which may be x or r itself
  uint16_t* y;      // bf16 result, or null
  int8_t* codes;    // 8-bit result, or null
  float* scales;
};

constexpr uint64_t kInf64 = 0x7FF0000000000000ull;

// kLanes lanes to a row (a part of a wave, a wave, or several), kHeld chunks of 8 columns a lane
// (kLanes * kHeld * 8 >= k); 4 waves a workgroup, or a row's.  A whole wave to rows of 128
// columns, as the norm of an attention's heads has them, would leave three lanes of four idle:
// 65,536 such rows to codes 17.1 us against 51.8.  The weights' chunks stay in registers over
// the rows of a workgroup, but for rows of more than 16384 columns: their registers hold t,
// and weights and residual come two chunks at a time (256 rows of 32768 to codes 18.2 us
// against 56.3 with everything held, which spills).
template <int kLanes>
struct NormShape {
  static constexpr int kTeam = kLanes > kWave ? kLanes / kWave : 1;  // waves to a row
  static constexpr int kWaves = kTeam > 4 ? kTeam : 4;
  static constexpr int kRows = kWaves * kWave / kLanes;  // rows at a time
};

template <int kLanes, int kHeld, bool kCodes>
__global__ __launch_bounds__(NormShape<kLanes>::kWaves* kWave) void rms_norm_kernel(NormArgs p) {
  constexpr int kTeam = NormShape<kLanes>::kTeam, kWaves = NormShape<kLanes>::kWaves, kRows = NormShape<kLanes>::kRows;
  constexpr int kPart = kLanes < kWave ? kLanes : kWave;
  constexpr bool kKeep = kLanes < 1024 || kHeld <= 2;
  constexpr int kGroup = kKeep ? kHeld : 2;  // chunks of the residual in flight
  __shared__ double s_sum[kTeam > 1 ? kWaves : 1];
  __shared__ uint64_t s_most[kTeam > 1 ? kWaves : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int part = wave % kTeam;
  const int j0 = (part * kWave + lane_id() % kPart) * 8;
  constexpr int kStep = kLanes * 8;
  const auto weight = [&](int c) { return *reinterpret_cast<const u16x8_t*>(p.w + min(j0 + c * kStep, p.k - 8)); };
  u16x8_t kept[kKeep ? kHeld : 1];
  bool large = false, looked = false;
  if constexpr (kKeep) {
#pragma unroll
    for (int c = 0; c < kHeld; ++c) kept[c] = weight(c);
  }
  const auto w = [&](int c) {
    if constexpr (kKeep) return kept[c];
    else return weight(c);
  };
  // Of a wave's rows the first: lanes whose own lies past the last one read the last and write
  // nothing, so that the whole wave takes part in what follows.
  for (int64_t first = (int64_t)blockIdx.x * kRows + (kLanes < kWave ? wave * (kWave / kPart) : wave / kTeam);
       first < p.rows; first += (int64_t)gridDim.x * kRows) {
    int64_t row = first;
    bool live = true;
    if constexpr (kLanes < kWave) {
      row = first + lane_id() / kPart;
      live = row < p.rows;
      row = min(row, p.rows - 1);
    }
    u16x8_t t[kHeld], r[kGroup];
    const int64_t at = row * p.k;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) t[c] = *reinterpret_cast<const u16x8_t*>(p.x + at + min(j0 + c * kStep, p.k - 8));
    if (p.r) {
#pragma unroll
      for (int g = 0; g < kHeld; g += kGroup) {
#pragma unroll
        for (int c = 0; c < kGroup; ++c)
          r[c] = *reinterpret_cast<const u16x8_t*>(p.r + at + min(j0 + (g + c) * kStep, p.k - 8));
#pragma unroll
        for (int c = 0; c < kGroup; ++c) {
          u16x8_t& v = t[g + c];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = i8_bf16(bf16_bits_to_f32(v[i]) + bf16_bits_to_f32(r[c][i]));
          if (live && j0 + (g + c) * kStep < p.k) *reinterpret_cast<u16x8_t*>(p.total + at + j0 + (g + c) * kStep) = v;
        }
      }
    }
    double sum = 0.0;
    uint64_t most = 0;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
      if (j0 + c * kStep >= p.k) continue;
      const u16x8_t wc = w(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = bf16_bits_to_f32(t[c][i]);
        sum = fma(v, v, sum);
        if constexpr (kCodes) {  // as bits: a NaN lies above infinity
          const double u = v * (double)bf16_bits_to_f32(wc[i]);
          most = max(most, (uint64_t)__double_as_longlong(u) & 0x7FFFFFFFFFFFFFFFull);
        }
      }
    }
    sum = wave_sum_f64<kPart>(sum);
    if constexpr (kCodes) most = wave_max_u64<kPart>(most);
    if constexpr (kTeam > 1) {
      if (lane_id() == 0) {
        s_sum[wave] = sum;
        if constexpr (kCodes) s_most[wave] = most;
      }
      lds_sync();
      sum = 0.0;
#pragma unroll
      for (int o = 0; o < kTeam; ++o) {
        sum += s_sum[wave - part + o];
        if constexpr (kCodes) most = max(most, s_most[wave - part + o]);
      }
      lds_sync();  // read before the next row's are written
    }
    const double root = sqrt(sum / p.k + p.eps), inv = 1.0 / root;
    if constexpr (!kCodes) {
      // Two fp32 roundings of 2^-24 before the one to bf16.  t * f may lie below 2^-126, where fp32 is
      // off by up to 2^-150; weights below 2^14 make that 2^-136 at most, an eighth of bf16's last bit.
      const float f = (float)inv;
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        const u16x8_t wc = w(c);
        u16x8_t o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i8_bf16(bf16_bits_to_f32(t[c][i]) * f * bf16_bits_to_f32(wc[i]));
        if (live && j0 + c * kStep < p.k) *reinterpret_cast<u16x8_t*>(p.y + at + j0 + c * kStep) = o;
      }
      if (!looked) {  // at the weights once, and here, where no row's loads wait for them
        u16x8_t most = {};
#pragma unroll
        for (int c = 0; c < kHeld; ++c) most = __builtin_elementwise_max(most, w(c) & (uint16_t)0x7FFF);
        large = __any(__builtin_reduce_max(most) >= 0x4680) != 0;  // 2^14
        looked = true;
      }
      // Larger weights, and a factor that is below 2^-126 itself, take fp64: again, from memory, so that
      // the registers are the ordinary rows'.
      if (large || f < 0x1p-126f) {
        const uint16_t* from = (p.r ? p.total : p.x) + at;
#pragma unroll 1
        for (int j = live ? j0 : p.k; j < p.k; j += j % 8 == 7 ? kStep - 7 : 1)
          p.y[at + j] = i8_bf16((float)((double)bf16_bits_to_f32(from[j]) * (double)bf16_bits_to_f32(p.w[j]) * inv));
      }
    } else {
      const bool bad = most >= kInf64 || !(sum < __longlong_as_double((long long)kInf64));
      const float scale = bad ? __uint_as_float(0x7FC00000u) : (float)(__longlong_as_double((long long)most) * inv / 127.0);
      const double per = scale > 0.0f ? inv / (double)scale : 0.0;  // zero and NaN scales: codes 0
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        const u16x8_t wc = w(c);
        uint32_t q[2] = {};
        u16x8_t o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double u = (double)bf16_bits_to_f32(t[c][i]) * (double)bf16_bits_to_f32(wc[i]);
          const int code = scale > 0.0f ? max(-127, min(127, (int)rint(u * per))) : 0;
          q[i / 4] |= (uint32_t)(code & 0xFF) << (8 * (i % 4));
          o[i] = i8_bf16((float)(u * inv));
        }
        if (live && j0 + c * kStep < p.k) {
          *reinterpret_cast<uint2*>(p.codes + at + j0 + c * kStep) = make_uint2(q[0], q[1]);
          if (p.y) *reinterpret_cast<u16x8_t*>(p.y + at + j0 + c * kStep) = o;
        }
      }
      if (live && part == 0 && lane_id() % kPart == 0) p.scales[row] = scale;
      // Quotients just between two codes, which one rounding moves off the border: rows of one magnitude have
      // them, whose root is short, and rows that eps rules, whose factor is 1 or 1000.  With a root of 29
      // bits at most root * scale is exact, with a factor of 37 u * inv, and one division decides (again,
      // from memory).
      const bool short_root = ((uint64_t)__double_as_longlong(root) & 0xFFFFFFu) == 0;
      if (scale > 0.0f && (short_root || ((uint64_t)__double_as_longlong(inv) & 0xFFFFu) == 0)) {
        const double times = short_root ? 1.0 : inv, step = short_root ? root * (double)scale : (double)scale;
        const uint16_t* from = (p.r ? p.total : p.x) + at;
#pragma unroll 1
        for (int j = live ? j0 : p.k; j < p.k; j += j % 8 == 7 ? kStep - 7 : 1) {
          const double u = (double)bf16_bits_to_f32(from[j]) * (double)bf16_bits_to_f32(p.w[j]);
          p.codes[at + j] = (int8_t)max(-127, min(127, (int)rint(u * times / step)));
        }
      }
    }
  }
}

template <int kLanes, int kHeld>
hipError_t launch_norm(const NormArgs& p, hipStream_t stream) {
  constexpr int kWaves = NormShape<kLanes>::kWaves, kRows = NormShape<kLanes>::kRows;
  // two workgroups' worth of waves a SIMD and more: the rest in turn, with the weights held
  const int64_t most = (int64_t)device_cu_count() * (32 / kWaves);
  const dim3 grid((unsigned)std::min<int64_t>((p.rows + kRows - 1) / kRows, most)), threads(kWaves * kWave);
  if (p.codes) hipLaunchKernelGGL((rms_norm_kernel<kLanes, kHeld, true>), grid, threads, 0, stream, p);
  else hipLaunchKernelGGL((rms_norm_kernel<kLanes, kHeld, false>), grid, threads, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t run_rms_norm(const uint16_t* x, const uint16_t* r, const uint16_t* w, int64_t rows, int k, double eps,
                        uint16_t* total, uint16_t* y, int8_t* codes, float* scales, hipStream_t stream) {
  const NormArgs p{x, r, w, rows, k, eps, total, y, codes, scales};
  // Up to two rows a compute unit: four waves to each, for the latency (2048 columns to codes:
  // 512 rows 4.8 us against 5.6 with a wave to each, 1 row 3.7 against 4.7).  More rows: a wave
  // to each, which needs no barrier (1024 rows 6.1 us against 6.9, 8192 rows of 1024 18.6
  // against 26.2).
  const bool few = rows <= 2 * (int64_t)device_cu_count();
  if (k <= 128) return launch_norm<16, 1>(p, stream);
  if (k <= 256) return launch_norm<32, 1>(p, stream);
  if (k <= 512) return launch_norm<64, 1>(p, stream);
  if (!few && k <= 1024) return launch_norm<64, 2>(p, stream);
  if (!few && k <= 2048) return launch_norm<64, 4>(p, stream);
  if (k <= 2048) return launch_norm<256, 1>(p, stream);
  if (k <= 4096) return launch_norm<256, 2>(p, stream);
  if (k <= 8192) return launch_norm<256, 4>(p, stream);
  if (k <= 16384) return launch_norm<1024, 2>(p, stream);
  if (k <= 32768) return launch_norm<1024, 4>(p, stream);
  return launch_norm<1024, 8>(p, stream);
}

}  // namespace q4moe
