// Root-mean-square norm of rows, with the residual's addition before it and a bf16 or an
// 8-bit result (rms_norm).
//
//   t = bf16(x + r)   y = t / sqrt(sum t^2 / k + eps) * w
//
// One pass: a row's t stay in registers between its sums and its results.  The sum of squares
// and what the codes' borders hang on (y, the largest |t w|, y / scale) are in fp64, so a
// code is the definition's: in fp32 about one code in 50,000 fell on the other side of a
// border.  The fp64 operations cost nothing beside the bytes: about ten an element, at a rate
// of 64 a clock and compute unit.
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

// kTeam waves to a row, kHeld chunks of 8 columns a lane (kTeam * kHeld * 512 >= k); 4 waves a
// workgroup, or kTeam.  The weights' chunks stay in registers over the rows of a workgroup.
template <int kTeam, int kHeld, bool kCodes>
__global__ __launch_bounds__(kTeam > 4 ? kTeam * kWave : 4 * kWave) void rms_norm_kernel(NormArgs p) {
  constexpr int kWaves = kTeam > 4 ? kTeam : 4, kRows = kWaves / kTeam;  // rows at a time
  __shared__ double s_sum[kTeam > 1 ? kWaves : 1];
  __shared__ uint64_t s_most[kTeam > 1 ? kWaves : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int part = wave % kTeam;
  const int j0 = (part * kWave + lane_id()) * 8;
  constexpr int kStep = kTeam * kWave * 8;
  u16x8_t w[kHeld];
#pragma unroll
  for (int c = 0; c < kHeld; ++c) w[c] = *reinterpret_cast<const u16x8_t*>(p.w + min(j0 + c * kStep, p.k - 8));
  for (int64_t row = (int64_t)blockIdx.x * kRows + wave / kTeam; row < p.rows; row += (int64_t)gridDim.x * kRows) {
    u16x8_t t[kHeld], r[kHeld];
    const int64_t at = row * p.k;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) t[c] = *reinterpret_cast<const u16x8_t*>(p.x + at + min(j0 + c * kStep, p.k - 8));
    if (p.r) {
#pragma unroll
      for (int c = 0; c < kHeld; ++c) r[c] = *reinterpret_cast<const u16x8_t*>(p.r + at + min(j0 + c * kStep, p.k - 8));
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[c][i] = i8_bf16(bf16_bits_to_f32(t[c][i]) + bf16_bits_to_f32(r[c][i]));
        if (j0 + c * kStep < p.k) *reinterpret_cast<u16x8_t*>(p.total + at + j0 + c * kStep) = t[c];
      }
    }
    double sum = 0.0;
    uint64_t most = 0;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
      if (j0 + c * kStep >= p.k) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = bf16_bits_to_f32(t[c][i]);
        sum = fma(v, v, sum);
        if constexpr (kCodes) {  // as bits: a NaN lies above infinity
          const double u = v * (double)bf16_bits_to_f32(w[c][i]);
          most = max(most, (uint64_t)__double_as_longlong(u) & 0x7FFFFFFFFFFFFFFFull);
        }
      }
    }
    sum = wave_sum_f64(sum);
    if constexpr (kCodes) most = wave_max_u64(most);
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
    const double inv = 1.0 / sqrt(sum / p.k + p.eps);
    if constexpr (!kCodes) {
      // two fp32 roundings of 2^-24 before the one to bf16
      const float f = (float)inv;
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        u16x8_t o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i8_bf16(bf16_bits_to_f32(t[c][i]) * f * bf16_bits_to_f32(w[c][i]));
        if (j0 + c * kStep < p.k) *reinterpret_cast<u16x8_t*>(p.y + at + j0 + c * kStep) = o;
      }
    } else {
      const bool bad = most >= kInf64 || !(sum < __longlong_as_double((long long)kInf64));
      const float scale = bad ? __uint_as_float(0x7FC00000u) : (float)(__longlong_as_double((long long)most) * inv / 127.0);
      const double per = scale > 0.0f ? inv / (double)scale : 0.0;  // zero and NaN scales: codes 0
#pragma unroll
      for (int c = 0; c < kHeld; ++c) {
        uint32_t q[2] = {};
        u16x8_t o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double u = (double)bf16_bits_to_f32(t[c][i]) * (double)bf16_bits_to_f32(w[c][i]);
          const int code = scale > 0.0f ? max(-127, min(127, (int)rint(u * per))) : 0;
          q[i / 4] |= (uint32_t)(code & 0xFF) << (8 * (i % 4));
          o[i] = i8_bf16((float)(u * inv));
        }
        if (j0 + c * kStep < p.k) {
          *reinterpret_cast<uint2*>(p.codes + at + j0 + c * kStep) = make_uint2(q[0], q[1]);
          if (p.y) *reinterpret_cast<u16x8_t*>(p.y + at + j0 + c * kStep) = o;
        }
      }
      if (part == 0 && lane_id() == 0) p.scales[row] = scale;
    }
  }
}

template <int kTeam, int kHeld>
hipError_t launch_norm(const NormArgs& p, hipStream_t stream) {
  constexpr int kWaves = kTeam > 4 ? kTeam : 4, kRows = kWaves / kTeam;
  // two workgroups' worth of waves a SIMD and more: the rest in turn, with the weights held
  const int64_t most = (int64_t)device_cu_count() * (32 / kWaves);
  const dim3 grid((unsigned)std::min<int64_t>((p.rows + kRows - 1) / kRows, most)), threads(kWaves * kWave);
  if (p.codes) hipLaunchKernelGGL((rms_norm_kernel<kTeam, kHeld, true>), grid, threads, 0, stream, p);
  else hipLaunchKernelGGL((rms_norm_kernel<kTeam, kHeld, false>), grid, threads, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t run_rms_norm(const uint16_t* x, const uint16_t* r, const uint16_t* w, int64_t rows, int k, double eps,
                        uint16_t* total, uint16_t* y, int8_t* codes, float* scales, hipStream_t stream) {
  const NormArgs p{x, r, w, rows, k, eps, total, y, codes, scales};
  // Few rows: four waves to each, for the latency.
  const bool few = rows <= 2 * (int64_t)device_cu_count();
  if (k <= 512) return launch_norm<1, 1>(p, stream);
  if (!few && k <= 1024) return launch_norm<1, 2>(p, stream);
  if (!few && k <= 2048) return launch_norm<1, 4>(p, stream);
  if (k <= 2048) return launch_norm<4, 1>(p, stream);
  if (k <= 4096) return launch_norm<4, 2>(p, stream);
  if (k <= 8192) return launch_norm<4, 4>(p, stream);
  if (k <= 16384) return launch_norm<16, 2>(p, stream);
  return launch_norm<16, 8>(p, stream);
}

}  // namespace q4moe
