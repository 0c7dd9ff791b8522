// 8-bit integer products of few rows, bound by the weights' bytes: i8_gemm on up to 16
// rows, and the experts' feed-forward of a decode step (moe_experts_i8 on few slots).
//
// A wave multiplies 16 weight rows with up to 16 tokens by v_mfma_i32_16x16x64_i8: operand
// A is the weight, row = lane % 16, 16 bytes of columns 16*(lane/16).. per lane, straight
// from memory to registers; operand B the tokens' codes, column = lane % 16, read from LDS
// in the same column order.  The sum of output row 4*(lane/16) + i for token lane % 16 ends
// in register i.  Fewer than 16 tokens leave columns of the product unused, which costs
// nothing here: the matrix cores take 1 KB of weights in 16 cycles a SIMD, many times the
// rate at which memory brings them.
#include <algorithm>

#include "int8.h"
#include "steps.h"

namespace q4moe {

namespace {

constexpr int kSmallWaves = 4;
constexpr int kBatch = 8;                 // weight loads in flight per wave and matrix: 512 columns
constexpr int kBatchCols = kBatch * 64;

// LDS image of up to 16 token rows: piece (16 columns) j of row r at ((j / 4) * 4 * m + (j % 4) * m + r) * 16,
// so that the 64 lanes of an operand read m consecutive pieces per column group.  Columns from
// K up to the next multiple of the batch hold zeros: loads past a row's end may then bring any
// bytes.
__device__ __forceinline__ int image_at(int col, int r, int m) { return ((col >> 4) * m + r) * 16 + (col & 15); }

// Quantizes a row of K values into row r of the image, by `parts` waves of which this is
// number `part` (parts = 1: meet does nothing): they meet once, to share their maxima.
// between() runs when the row's loads are on their way: what it loads arrives behind them
// and meanwhile the codes are made.
template <int kHeld, typename In, typename Between, typename Meet>
__device__ __forceinline__ float quantize_row(const In* x, int K, int Kpad, uint8_t* image, int r, int m, int part,
                                              int parts, Between between, Meet meet) {
  const int lane = lane_id();
  // kHeld chunks of 8 values per lane stay in registers between the two passes, others are read again
  const int j0 = (part * kWave + lane) * 8, step = parts * kWave * 8;
  I8Chunk<In> held[kHeld];
#pragma unroll
  for (int c = 0; c < kHeld; ++c) held[c].load(x + min(j0 + c * step, K - 8));
  __builtin_amdgcn_sched_barrier(0);
  between();
  __builtin_amdgcn_sched_barrier(0);
  uint32_t most = 0;
#pragma unroll
  for (int c = 0; c < kHeld; ++c) most = held[c].most(most);
  for (int j = j0 + kHeld * step; j < K; j += step) {
    I8Chunk<In> v;
    v.load(x + j);
    most = v.most(most);
  }
  const float scale = i8_scale(meet(wave_max_u32(most)));
  const I8Rounder rd(scale);
  auto put = [&](int j, const I8Chunk<In>& v) { *reinterpret_cast<uint2*>(image + image_at(j, r, m)) = v.codes(rd); };
#pragma unroll
  for (int c = 0; c < kHeld; ++c) {
    if (j0 - lane * 8 + c * step >= K) break;  // uniform: the rest holds nothing of the row
    if (j0 + c * step < K) put(j0 + c * step, held[c]);
  }
  for (int j = j0 + kHeld * step; j < K; j += step) {
    I8Chunk<In> v;
    v.load(x + j);
    put(j, v);
  }
  for (int j = K + j0; j < Kpad; j += step)
    *reinterpret_cast<uint2*>(image + image_at(j, r, m)) = make_uint2(0u, 0u);
  return scale;
}

// A workgroup's m rows into the image: one wave a row, or for fewer than four rows two or
// four waves a row.  row(r) is row r's address; every wave passes the same barriers.
template <int kHeld, typename Row, typename Between>
__device__ __forceinline__ void quantize_rows(Row row, int m, int K, int Kpad, uint8_t* image, float* s_scale,
                                              uint32_t* s_most, Between between) {
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int parts = m == 1 ? kSmallWaves : m < kSmallWaves ? kSmallWaves / 2 : 1;
  const int part = wave % parts, at_once = kSmallWaves / parts;
  for (int r0 = 0; r0 < m; r0 += at_once) {
    const int r = min(r0 + wave / parts, m - 1);  // rows past the last repeat it
    auto meet = [&](uint32_t most) -> uint32_t {
      if (parts == 1) return most;
      if (lane == 0) s_most[wave] = most;
      lds_sync();
      const int first = wave - part;
      most = max(s_most[first], s_most[first + 1]);
      if (parts == kSmallWaves) most = max(most, max(s_most[2], s_most[3]));
      return most;
    };
    float scale;
    if (r0 == 0) scale = quantize_row<kHeld>(row(r), K, Kpad, image, r, m, part, parts, between, meet);
    else scale = quantize_row<kHeld>(row(r), K, Kpad, image, r, m, part, parts, [] {}, meet);
    if (lane == 0) s_scale[r] = scale;
    if (parts > 1 && r0 + at_once < m) lds_sync();  // s_most is read before the next rows' maxima
  }
  lds_sync();
}

// Rows that are codes already into the image, by the workgroup.
__device__ __forceinline__ void copy_rows(const int8_t* X, const float* Xs, int m, int K, int Kpad, uint8_t* image,
                                          float* s_scale) {
  const int per = Kpad / 16;  // pieces of a row
  for (int i = threadIdx.x; i < m * per; i += kSmallWaves * kWave) {
    const int r = i / per, col = (i - r * per) * 16;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (col < K) v = *reinterpret_cast<const uint4*>(X + (int64_t)r * K + col);
    *reinterpret_cast<uint4*>(image + image_at(col, r, m)) = v;
  }
  if (threadIdx.x < (unsigned)m) s_scale[threadIdx.x] = Xs[threadIdx.x];
  lds_sync();
}

// A batch of weight pieces of one row per lane: columns c0 + 64 j + 16 * (lane / 16), clamped to the row.
__device__ __forceinline__ void load_batch(const int8_t* row, int c0, int K, i32x4_t (&w)[kBatch]) {
  const int g = (lane_id() >> 4) * 16;
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    w[j] = *reinterpret_cast<const i32x4_t*>(row + min(c0 + j * 64 + g, K - 16));
}

typedef int i32x4acc_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4acc_t mul_batch(const i32x4_t (&w)[kBatch], const uint8_t* image, int c0, int m,
                                               i32x4acc_t acc) {
  const int lane = lane_id();
  const int r = min(lane & 15, m - 1);
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const i32x4_t x = *reinterpret_cast<const i32x4_t*>(image + image_at(c0 + j * 64 + (lane >> 4) * 16, r, m));
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x, acc, 0, 0, 0);
  }
  return acc;
}

// ---- i8_gemm on m <= 16 rows
// Measured: 8 rows on 151,936 x 2048 in 58-64 us (5.0 TB/s of the 317 MB; a large copy runs at
// 5.1), 1 row on 1024 x 2048 in 4.3 us (a launch and two memory latencies). Four workgroups on
// a compute unit: 64.5 us against 67.0 with two.
// Split: a workgroup per 16 weight rows, its waves share the columns (few rows: every
// compute unit gets some).  Otherwise each wave takes whole blocks of 16 rows in turn, with
// the next batch's loads in flight while one is multiplied.
// In: bf16 rows (uint16_t), or codes (int8_t) whose scales are sx.
template <bool kSplit, bool kBf16, typename In>
__global__ __launch_bounds__(kSmallWaves* kWave) void i8_few_rows_kernel(I8Mat W, int64_t n, int K,
                                                                         const In* __restrict__ X,
                                                                         const float* __restrict__ Xs, int m,
                                                                         void* __restrict__ Y) {
  extern __shared__ __align__(16) uint8_t s_image[];
  __shared__ float s_scale[16];
  __shared__ uint32_t s_most[kSmallWaves];
  __shared__ i32x4acc_t s_sum[kSplit ? kSmallWaves : 1][kWave];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int Kpad = (K + kBatchCols - 1) / kBatchCols * kBatchCols;
  const int batches = Kpad / kBatchCols;
  const int64_t blocks = (n + 15) / 16;
  const int64_t first = kSplit ? blockIdx.x : (int64_t)blockIdx.x * kSmallWaves + wave;
  const int64_t stride = kSplit ? gridDim.x : (int64_t)gridDim.x * kSmallWaves;
  const int b0 = kSplit ? wave : 0, bstep = kSplit ? kSmallWaves : 1;
  auto row_of = [&](int64_t blk) { return W.codes + min(blk * 16 + (lane & 15), n - 1) * K; };

  // the first weights are on their way while the rows are quantized
  i32x4_t w[kBatch];
  auto weights = [&] {
    if (first < blocks && b0 < batches) load_batch(row_of(first), b0 * kBatchCols, K, w);
  };
  if constexpr (sizeof(In) == 1) {
    weights();
    copy_rows(X, Xs, m, K, Kpad, s_image, s_scale);
  } else {
    quantize_rows<4>([&](int r) { return X + (int64_t)r * K; }, m, K, Kpad, s_image, s_scale, s_most, weights);
  }

  const int t = lane & 15;
  const float sx = s_scale[min(t, m - 1)];
  for (int64_t blk = first; blk < blocks; blk += stride) {
    i32x4acc_t acc = {};
    const int64_t next = blk + stride;
    for (int b = b0; b < batches; b += bstep) {
      i32x4_t nw[kBatch];
      const bool more = b + bstep < batches;
      if (more || next < blocks)
        load_batch(row_of(more ? blk : next), (more ? b + bstep : b0) * kBatchCols, K, nw);
      acc = mul_batch(w, s_image, b * kBatchCols, m, acc);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) w[j] = nw[j];
    }
    if constexpr (kSplit) {
      s_sum[wave][lane] = acc;
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int o = 1; o < kSmallWaves; ++o) acc += s_sum[o][lane];
      }
    }
    if ((!kSplit || wave == 0) && t < m) {
      const int64_t r0 = blk * 16 + (lane >> 4) * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r0 + i >= n) break;
        const float y = (float)acc[i] * sx * W.scales[r0 + i];
        if constexpr (kBf16) static_cast<uint16_t*>(Y)[t * n + r0 + i] = i8_bf16(y);
        else static_cast<float*>(Y)[t * n + r0 + i] = y;
      }
    }
    if constexpr (kSplit) __syncthreads();
  }
}

constexpr size_t kSmallLds = 64 * 1024;  // of codes: two workgroups or more share a compute unit

size_t image_bytes(int64_t m, int K) { return (size_t)m * ((K + kBatchCols - 1) / kBatchCols * kBatchCols); }

}  // namespace

bool i8_few_rows(int64_t m, int K) { return m <= 16 && image_bytes(m, K) <= kSmallLds; }

namespace {

template <typename In>
hipError_t launch_few_rows(const I8Mat& W, int64_t n, int K, const In* X, const float* Xs, int m, void* Y, int out_bf16,
                           hipStream_t stream) {
  const size_t lds = image_bytes(m, K);
  const int64_t blocks = (n + 15) / 16;
  const int64_t resident = 4 * (int64_t)device_cu_count();
  const bool split = blocks <= resident;
  const dim3 grid((unsigned)(split ? blocks : std::min<int64_t>(resident, (blocks + kSmallWaves - 1) / kSmallWaves)));
  const dim3 threads(kSmallWaves * kWave);
  if (split && out_bf16)
    hipLaunchKernelGGL((i8_few_rows_kernel<true, true, In>), grid, threads, lds, stream, W, n, K, X, Xs, m, Y);
  else if (split)
    hipLaunchKernelGGL((i8_few_rows_kernel<true, false, In>), grid, threads, lds, stream, W, n, K, X, Xs, m, Y);
  else if (out_bf16)
    hipLaunchKernelGGL((i8_few_rows_kernel<false, true, In>), grid, threads, lds, stream, W, n, K, X, Xs, m, Y);
  else
    hipLaunchKernelGGL((i8_few_rows_kernel<false, false, In>), grid, threads, lds, stream, W, n, K, X, Xs, m, Y);
  return hipGetLastError();
}

}  // namespace

hipError_t run_i8_few_rows(const I8Mat& W, int64_t n, int K, const uint16_t* X, int m, void* Y, int out_bf16,
                           hipStream_t stream) {
  return launch_few_rows(W, n, K, X, nullptr, m, Y, out_bf16, stream);
}

hipError_t run_i8_few_rows(const I8Mat& W, int64_t n, int K, const int8_t* codes, const float* scales, int m, void* Y,
                           int out_bf16, hipStream_t stream) {
  return launch_few_rows(W, n, K, codes, scales, m, Y, out_bf16, stream);
}

// ---- the experts' feed-forward on few slots, two launches
namespace {

// Slots of the step: t * k + i for a token's i-th expert, then P + t for token t's shared expert.
// Gate/up: a workgroup per (slot, 8 intermediate columns): the 16 rows of its operand are 8
// rows of gate and the same 8 of up, its four waves share the columns.  The first slot of an
// expert takes all slots of that expert (up to 16 at a time), the others leave.
// Measured at hidden 2048, intermediate 512, 8 of 256 experts and a shared one: one token 8 us
// (19 MB, latencies) and 5 us down; eight tokens 31 us for 122 MB (3.9 TB/s) and 18 us for 61
// MB (3.4 TB/s): what misses to the copy's 5.1 is the time in which workgroups quantize, meet
// and store while no loads of theirs are in flight. Two blocks of 8 columns a workgroup, with
// twice the loads in flight but half the workgroups, took 57 us for both against 54.
constexpr int kMaxSlots = 64;
constexpr int kUpCols = 8;

__global__ __launch_bounds__(kSmallWaves* kWave) void i8_slots_up_kernel(I8Experts L, const uint16_t* __restrict__ X,
                                                                         int T, int k, const int32_t* __restrict__ ids,
                                                                         float* __restrict__ act) {
  extern __shared__ __align__(16) uint8_t s_image[];
  __shared__ float s_scale[16];
  __shared__ uint32_t s_most[kSmallWaves];
  __shared__ i32x4acc_t s_sum[kSmallWaves][kWave];
  __shared__ int s_slot[kMaxSlots];  // i8_few_slots: no more, nor more than 16 tokens
  __shared__ int s_count[kSmallWaves];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int H = L.hidden, I = L.inter, P = T * k;
  const int slot0 = blockIdx.y;
  const int n0 = blockIdx.x * kUpCols;
  const bool sh = slot0 >= P;  // the shared expert's workgroups take every token
  const int e = sh ? 0 : ids[slot0];
  if (e < 0 || e >= L.n_experts) return;
  int count = 1;
  if (T > 1) {  // one token's slots are each their own
    const int mine = threadIdx.x;
    const bool same = sh ? mine < T : mine < P && ids[mine] == e;
    const uint64_t ball = __ballot(same);
    if (lane == 0) s_count[wave] = __popcll(ball);
    lds_sync();
    int base = 0;
    count = 0;
#pragma unroll
    for (int o = 0; o < kSmallWaves; ++o) {
      base += o < wave ? s_count[o] : 0;
      count += s_count[o];
    }
    if (same) s_slot[base + __popcll(ball & ((1ull << lane) - 1ull))] = sh ? P + mine : mine;
    lds_sync();
    if (s_slot[0] != slot0) return;  // uniform: an earlier slot has the same expert
  }
  auto slot_of = [&](int i) { return T > 1 ? s_slot[i] : slot0; };

  const int Kpad = (H + kBatchCols - 1) / kBatchCols * kBatchCols;
  const int batches = Kpad / kBatchCols;
  const I8Mat gate = sh ? L.sh_gate : L.gate, up = sh ? L.sh_up : L.up;
  const int64_t r0 = (int64_t)e * I + n0;
  const int a = lane & 15;
  const int8_t* row = (a < kUpCols ? gate.codes : up.codes) + (r0 + a % kUpCols) * H;
  // thread (token, column) of the result: its channels' scales are loaded with the weights
  const int col = threadIdx.x % kUpCols, tok = threadIdx.x / kUpCols;
  float sg = 0.f, su = 0.f;
  for (int s0 = 0; s0 < count; s0 += 16) {
    const int m = min(16, count - s0);
    if (s0 > 0) __syncthreads();  // the image and the sums are read no more
    i32x4_t w[kBatch];
    quantize_rows<1>(  // a lone row, the usual case, is one chunk a wave up to 2,048 columns
        [&](int r) {
          const int s = slot_of(s0 + r);
          return X + (int64_t)(s >= P ? s - P : s / k) * H;
        },
        m, H, Kpad, s_image, s_scale, s_most, [&] {
          if (wave < batches) load_batch(row, wave * kBatchCols, H, w);
          if (tok < m) {
            sg = gate.scales[r0 + col];
            su = up.scales[r0 + col];
          }
        });
    i32x4acc_t acc = {};
    for (int b = wave; b < batches; b += kSmallWaves) {
      if (b > wave) load_batch(row, b * kBatchCols, H, w);
      acc = mul_batch(w, s_image, b * kBatchCols, m, acc);
    }
    s_sum[wave][lane] = acc;
    __syncthreads();
    if (tok < m) {
      // operand row c of token t lies in lane 16 * (c / 4) + t, register c % 4
      int g = 0, u = 0;
#pragma unroll
      for (int o = 0; o < kSmallWaves; ++o) {
        g += s_sum[o][(col / 4) * 16 + tok][col % 4];
        u += s_sum[o][((col + kUpCols) / 4) * 16 + tok][col % 4];
      }
      const float sx = s_scale[tok];
      act[(int64_t)slot_of(s0 + tok) * I + n0 + col] = i8_swiglu(i8_scaled((float)g, sx, sg), i8_scaled((float)u, sx, su));
    }
  }
}

// Down and the weighted sum: a workgroup per (token, 16 output columns), a wave per slot
// (in turn).  kHalves: 8 output columns, their rows twice in the operand's 16, with the lower
// half of K and with the upper; the codes' halves stand as two tokens, and a sum is row r of
// the one plus row r + 8 of the other.  That puts one token's step on twice as many compute
// units: with hidden 2048 (128 workgroups of 16 columns) a step takes 12.6 us instead of 13.0.
// It is for one token whose blocks of 16 are fewer than the compute units, and intermediate
// sizes whose halves are whole batches of loads.
template <bool kHalves>
__global__ void i8_slots_down_kernel(I8Experts L, int T, int k, const int32_t* __restrict__ ids,
                                     const float* __restrict__ weights, int shared, const float* __restrict__ act,
                                     void* __restrict__ Y, int out_bf16) {
  extern __shared__ __align__(16) uint8_t s_dyn[];  // [waves] images of one row, then [slots][kCols] parts
  constexpr int kCols = kHalves ? 8 : 16;
  constexpr int kLoads = kHalves ? kBatch / 2 : kBatch;  // 64 columns each
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int H = L.hidden, I = L.inter, P = T * k, slots = k + shared;
  const int t = blockIdx.y;
  const int n0 = blockIdx.x * kCols;
  const int Kpad = (I + kBatchCols - 1) / kBatchCols * kBatchCols;
  const int K = kHalves ? I / 2 : I;  // columns that a lane's operand row covers (halves: a multiple of 256)
  uint8_t* image = s_dyn + (size_t)wave * Kpad;
  float* s_part = reinterpret_cast<float*>(s_dyn + (size_t)waves * Kpad);
  const int a = lane & 15, g = (lane >> 4) * 16;
  const int w_row = a % kCols, w_col = kHalves ? (a / kCols) * K : 0;  // this lane's weight row and first column
  const uint8_t* codes = image + (kHalves ? (lane & 1) * K : 0) + g;   // and its codes (one row: column c at c)
  for (int s = wave; s < slots; s += waves) {
    const bool sh = s >= k;
    const int e = sh ? 0 : ids[t * k + s];
    const bool there = e >= 0 && e < L.n_experts;
    float v[4] = {};
    if (there) {
      const I8Mat down = sh ? L.sh_down : L.down;
      const int64_t r0 = (int64_t)e * H + n0;
      const int8_t* row = down.codes + (r0 + w_row) * I + w_col;
      const int64_t slot = sh ? P + t : t * k + s;
      const int out_row = (lane >> 4) * 4 % kCols;  // output columns out_row .. + 3 of this lane
      i32x4_t w[kLoads];
      auto load = [&](int c) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          w[j] = *reinterpret_cast<const i32x4_t*>(row + min(c + j * 64 + g, K - 16));
      };
      float sw[4], f = 1.0f;
      const float scale = quantize_row<1>(
          act + slot * I, I, Kpad, image, 0, 1, 0, 1,
          [&] {
            load(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) sw[i] = down.scales[r0 + out_row + i];
            if (!sh) f = weights[t * k + s];
          },
          [](uint32_t most) { return most; });
      __builtin_amdgcn_wave_barrier();
      i32x4acc_t acc = {};
      for (int c = 0; c < K; c += kLoads * 64) {
        if (c > 0) load(c);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], *reinterpret_cast<const i32x4_t*>(codes + c + j * 64), acc,
                                                      0, 0, 0);
      }
      if constexpr (kHalves) {
        // rows 0..7 of token 0 lie in lanes 0 and 16, rows 8..15 of token 1 in lanes 33 and 49
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += __shfl(acc[i], lane + 33, kWave);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = i8_scaled((float)acc[i], scale, sw[i]) * f;
      __builtin_amdgcn_wave_barrier();  // the image is read before the next slot's replaces it
    }
    if (a == 0 && (lane >> 4) * 4 < kCols)
      *reinterpret_cast<float4*>(s_part + s * kCols + (lane >> 4) * 4) = make_float4(v[0], v[1], v[2], v[3]);
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    float y = 0.f;
    for (int s = 0; s < slots; ++s) y += s_part[s * kCols + threadIdx.x];
    const int64_t at = (int64_t)t * H + n0 + threadIdx.x;
    if (out_bf16) static_cast<uint16_t*>(Y)[at] = i8_bf16(y);
    else static_cast<float*>(Y)[at] = y;
  }
}

int down_waves(int I, int slots) {
  const int Kpad = (I + kBatchCols - 1) / kBatchCols * kBatchCols;
  return std::max(1, std::min({slots, 16, (int)(kSmallLds / Kpad)}));
}

}  // namespace

// Up to 64 slots: one token 13 us against the grouped form's 39, 64 slots over 256 experts
// 54 against 69 and over 16 experts 41 against 40; at 128 slots the two are level (97 and 99
// us over 256 experts) and more tokens share an expert's rows in the grouped form.
bool i8_few_slots(const I8Experts& L, int64_t T, int k) {
  return T * k <= 64 && T <= 16 && image_bytes(T * k < 16 ? T * k : 16, L.hidden) <= kSmallLds;
}

size_t i8_few_slots_bytes(const I8Experts& L, int64_t T, int k) {
  return (size_t)(T * k + (L.sh_gate.codes ? T : 0)) * L.inter * 4;
}

hipError_t run_i8_few_slots(const I8Experts& L, const uint16_t* X, int T, const int32_t* ids, const float* weights,
                            int k, void* Y, int out_bf16, float* act, hipStream_t stream) {
  const int shared = L.sh_gate.codes ? 1 : 0, P = T * k;
  const int m = std::min(std::max(P, T), 16);
  hipLaunchKernelGGL(i8_slots_up_kernel, dim3(L.inter / kUpCols, P + shared), dim3(kSmallWaves * kWave),
                     image_bytes(m, L.hidden), stream, L, X, T, k, ids, act);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int waves = down_waves(L.inter, k + shared);
  const size_t lds = (size_t)waves * ((L.inter + kBatchCols - 1) / kBatchCols * kBatchCols) + (size_t)(k + shared) * 64;
  const dim3 threads(waves * kWave);
  if (T == 1 && L.inter % kBatchCols == 0 && L.hidden / 16 < device_cu_count())
    hipLaunchKernelGGL(i8_slots_down_kernel<true>, dim3(L.hidden / 8, T), threads, lds, stream, L, T, k, ids, weights,
                       shared, act, Y, out_bf16);
  else
    hipLaunchKernelGGL(i8_slots_down_kernel<false>, dim3(L.hidden / 16, T), threads, lds, stream, L, T, k, ids, weights,
                       shared, act, Y, out_bf16);
  return hipGetLastError();
}

}  // namespace q4moe
