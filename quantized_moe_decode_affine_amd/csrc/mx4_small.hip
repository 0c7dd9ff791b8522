// Microscaled 4-bit products of few rows, bound by the weights' bytes: mx4_gemm on up to 16
// rows, and the experts' feed-forward of a decode step (moe_experts_mx4 on few slots).
//
// A wave multiplies 16 weight rows with up to 16 tokens by v_mfma_scale_f32_16x16x128_f8f6f4:
// operand A is the weight, row = lane % 16, 32 columns (16 bytes) from 32*(lane/16), straight
// from memory to registers; operand B the tokens' codes, column = lane % 16, read from LDS in
// the same column order.  The sum of output row 4*(lane/16) + i for token lane % 16 ends in
// register i.  Fewer than 16 tokens leave columns of the product unused, which costs nothing
// here: the matrix cores take 1 KB of weights in 16 cycles a SIMD, many times the rate at
// which memory brings them.
//
// Measured: 8 rows on 151936 x 2048 (165 MB of weights and 5 of results) 29 us where the last cache
// holds a part of the weights from the call before, 5.8 TB/s; a call after others 37 us, 4.6 TB/s.
// 1 row on 1024 x 2048 in 3.5 us, a launch and two turns of memory; experts of one token (8 of 256
// and a shared one, 2048 x 512) 5.0 us for gate and up and 4.4 for down, traced apart; 8.7 the two
// in a graph.
#include <algorithm>

#include "steps.h"
#include "mx4.h"

namespace q4moe {

namespace {

constexpr int kSmallWaves = 4;
constexpr int kBatch = 4;                   // weight loads in flight per wave and operand: 512 columns
constexpr int kBatchCols = kBatch * 128;
constexpr int kBatchScales = kBatchCols / kMxBlock;  // 16 bytes a row

int padded(int K) { return (K + kBatchCols - 1) / kBatchCols * kBatchCols; }

// LDS image of up to 16 token rows.  Codes: piece (32 columns) j of row r at (j * m + r) * 16,
// so that the 64 lanes of an operand read m consecutive pieces per column group; then the
// scales, row by row.  Columns from K up to the next multiple of the batch hold zeros, so
// loads of weights past a row's end may bring any bytes there.
struct Image {
  uint8_t* codes;   // m * Kpad / 2 bytes
  uint8_t* scales;  // m * Kpad / 32
  int m, Kpad;
  __device__ __forceinline__ Image(uint8_t* base, int m_, int Kpad_)
      : codes(base), scales(base + m_ * (Kpad_ / 2)), m(m_), Kpad(Kpad_) {}
  __device__ __forceinline__ i32x4_t operand(int piece, int r) const {
    return *reinterpret_cast<const i32x4_t*>(codes + (piece * m + r) * 16);
  }
  __device__ __forceinline__ uint4 batch_scales(int c0, int r) const {
    return *reinterpret_cast<const uint4*>(scales + r * (Kpad / kMxBlock) + c0 / kMxBlock);
  }
};
size_t image_bytes(int64_t m, int K) { return (size_t)m * (padded(K) / 2 + padded(K) / kMxBlock); }

// Rows of K values into the image, by `threads` threads of which this is number `tid` (a
// multiple of 64 of them).  row(r) is row r's address.  between() runs when the first loads
// are on their way.
template <typename In, typename Row, typename Between>
__device__ __forceinline__ void fill_image(const Image& im, Row row, int K, int tid, int threads, Between between) {
  const int per = im.Kpad / 16, total = im.m * per;  // halves of blocks: an even number of them a row
  bool first = true;
  for (int i = tid; i - tid % kWave < total; i += threads) {
    const int r = min(i / per, im.m - 1), col = (i - r * per) * 16;  // both lanes of a block agree
    Mx4Half<In> v;
    if (i < total && col < K) v.load(row(r) + col);
    if (first) {
      __builtin_amdgcn_sched_barrier(0);
      between();
      __builtin_amdgcn_sched_barrier(0);
      first = false;
    }
    if (i < total) {
      uint32_t byte = 0;
      uint2 c = make_uint2(0u, 0u);
      if (col < K) c = v.codes(&byte);
      *reinterpret_cast<uint2*>(im.codes + ((col >> 5) * im.m + r) * 16 + (col & 16) / 2) = c;
      if ((col & 16) == 0) im.scales[r * (im.Kpad / kMxBlock) + (col >> 5)] = (uint8_t)byte;
    }
  }
  if (first) between();
}

// A batch of one weight row per lane: codes of columns c0 + 128 j + 32 * (lane / 16), and the
// scales of its 16 blocks (the same for the four lanes of a row).  What would lie past the
// row's end is read from its last columns.
struct WeightBatch {
  i32x4_t w[kBatch];
  uint4 scales;
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* sc, int c0, int K) {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      w[j] = *reinterpret_cast<const i32x4_t*>(codes + min(c0 / 2 + j * 64 + g * 16, K / 2 - 16));
    const int at = c0 / kMxBlock, last = K / kMxBlock - 2;
    if (at + kBatchScales - 2 <= last) {
      __builtin_memcpy(&scales, sc + at, 16);
    } else {
      uint32_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d[j] = *reinterpret_cast<const uint16_t*>(sc + min(at + 4 * j, last)) |
               (uint32_t)*reinterpret_cast<const uint16_t*>(sc + min(at + 4 * j + 2, last)) << 16;
      scales = make_uint4(d[0], d[1], d[2], d[3]);
    }
  }
};

__device__ __forceinline__ f32x4_t mul_batch(const WeightBatch& b, const Image& im, int c0, f32x4_t acc) {
  const int lane = lane_id(), g = lane >> 4;
  const int r = min(lane & 15, im.m - 1);
  const uint4 xs = im.batch_scales(c0, r);
  const uint32_t x[4] = {xs.x, xs.y, xs.z, xs.w}, w[4] = {b.scales.x, b.scales.y, b.scales.z, b.scales.w};
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const i32x4_t v = im.operand(c0 / kMxBlock + 4 * j + g, r);
    // a lane's scale is byte g of the four blocks' word
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4_operand(b.w[j]), mx4_operand(v), acc, kFp4, kFp4, 0,
                                                           (int)(w[j] >> (8 * g)), 0, (int)(x[j] >> (8 * g)));
  }
  return acc;
}

// ---- mx4_gemm on m <= 16 rows
// Against the tiles: 16 rows on 1024 x 2048 7.2 us to 10.2, on 151936 x 2048 34.6 to 37.5.
// Split: a workgroup per 16 weight rows, its waves share the columns (few rows: every
// compute unit gets some).  Otherwise each wave takes whole blocks of 16 rows in turn, with
// the next batch's loads in flight while one is multiplied (two of them: 151936 x 2048 on 8
// rows 35.9 us for 37.0, on 1 row 32.7 for 31.3; three spill).
template <bool kSplit, bool kBf16>
__global__ __launch_bounds__(kSmallWaves* kWave) void mx4_few_rows_kernel(Mx4Mat W, int64_t n, int K,
                                                                          const uint16_t* __restrict__ X, int m,
                                                                          void* __restrict__ Y) {
  extern __shared__ __align__(16) uint8_t s_image[];
  __shared__ f32x4_t s_sum[kSplit ? kSmallWaves : 1][kWave];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const Image im(s_image, m, (K + kBatchCols - 1) / kBatchCols * kBatchCols);
  const int batches = im.Kpad / kBatchCols;
  const int64_t blocks = (n + 15) / 16;
  const int64_t first = kSplit ? blockIdx.x : (int64_t)blockIdx.x * kSmallWaves + wave;
  const int64_t stride = kSplit ? gridDim.x : (int64_t)gridDim.x * kSmallWaves;
  const int b0 = kSplit ? wave : 0, bstep = kSplit ? kSmallWaves : 1;
  auto load = [&](WeightBatch& w, int64_t blk, int b) {
    const int64_t row = min(blk * 16 + (lane & 15), n - 1);
    w.load(W.codes + row * (K / 2), W.scales + row * (K / kMxBlock), b * kBatchCols, K);
  };

  // the first weights are on their way while the rows are quantized
  WeightBatch w;
  fill_image<uint16_t>(im, [&](int r) { return X + (int64_t)r * K; }, K, threadIdx.x, kSmallWaves * kWave, [&] {
    if (first < blocks && b0 < batches) load(w, first, b0);
  });
  lds_sync();

  const int t = lane & 15;
  for (int64_t blk = first; blk < blocks; blk += stride) {
    f32x4_t acc = {};
    const int64_t next = blk + stride;
    for (int b = b0; b < batches; b += bstep) {
      WeightBatch nw;
      const bool more = b + bstep < batches;
      if (more || next < blocks) load(nw, more ? blk : next, more ? b + bstep : b0);
      acc = mul_batch(w, im, b * kBatchCols, acc);
      w = nw;
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
        if constexpr (kBf16) static_cast<uint16_t*>(Y)[t * n + r0 + i] = i8_bf16(acc[i]);
        else static_cast<float*>(Y)[t * n + r0 + i] = acc[i];
      }
    }
    if constexpr (kSplit) __syncthreads();
  }
}

constexpr size_t kSmallLds = 64 * 1024;  // of codes: two workgroups or more share a compute unit

}  // namespace

bool mx4_few_rows(int64_t m, int K) { return m <= 16 && image_bytes(m, K) <= kSmallLds; }

hipError_t run_mx4_few_rows(const Mx4Mat& W, int64_t n, int K, const uint16_t* X, int m, void* Y, int out_bf16,
                            hipStream_t stream) {
  const size_t lds = image_bytes(m, K);
  const int64_t blocks = (n + 15) / 16;
  const int64_t resident = 4 * (int64_t)device_cu_count();
  const bool split = blocks <= resident;
  const dim3 grid((unsigned)(split ? blocks : std::min<int64_t>(resident, (blocks + kSmallWaves - 1) / kSmallWaves)));
  const dim3 threads(kSmallWaves * kWave);
  if (split && out_bf16)
    hipLaunchKernelGGL((mx4_few_rows_kernel<true, true>), grid, threads, lds, stream, W, n, K, X, m, Y);
  else if (split)
    hipLaunchKernelGGL((mx4_few_rows_kernel<true, false>), grid, threads, lds, stream, W, n, K, X, m, Y);
  else if (out_bf16)
    hipLaunchKernelGGL((mx4_few_rows_kernel<false, true>), grid, threads, lds, stream, W, n, K, X, m, Y);
  else
    hipLaunchKernelGGL((mx4_few_rows_kernel<false, false>), grid, threads, lds, stream, W, n, K, X, m, Y);
  return hipGetLastError();
}

// ---- the experts' feed-forward on few slots, two launches
namespace {

// Slots of the step: t * k + i for a token's i-th expert, then P + t for token t's shared expert.
// Gate/up: a workgroup per (slot, 8 intermediate columns): the 16 rows of its operand are 8
// rows of gate and the same 8 of up, its four waves share the columns.  The first slot of an
// expert takes all slots of that expert (up to 16 at a time), the others leave.
constexpr int kMaxSlots = 128;  // (at most the workgroup's threads, 256)
constexpr int kUpCols = 8;

__global__ __launch_bounds__(kSmallWaves* kWave) void mx4_slots_up_kernel(Mx4Experts L, const uint16_t* __restrict__ X,
                                                                          int T, int k, const int32_t* __restrict__ ids,
                                                                          float* __restrict__ act) {
  extern __shared__ __align__(16) uint8_t s_image[];
  __shared__ f32x4_t s_sum[kSmallWaves][kWave];
  __shared__ int s_slot[kMaxSlots];
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
  const Mx4Mat gate = sh ? L.sh_gate : L.gate, up = sh ? L.sh_up : L.up;
  const int64_t r0 = (int64_t)e * I + n0;
  const int a = lane & 15;
  const Mx4Mat own = a < kUpCols ? gate : up;
  const uint8_t* row = own.codes + (r0 + a % kUpCols) * (H / 2);
  const uint8_t* row_scales = own.scales + (r0 + a % kUpCols) * (H / kMxBlock);
  const int col = threadIdx.x % kUpCols, tok = threadIdx.x / kUpCols;  // thread (token, column) of the result
  for (int s0 = 0; s0 < count; s0 += 16) {
    const int m = min(16, count - s0);
    if (s0 > 0) __syncthreads();  // the image and the sums are read no more
    const Image im(s_image, m, Kpad);
    WeightBatch w;
    fill_image<uint16_t>(
        im,
        [&](int r) {
          const int s = slot_of(s0 + r);
          return X + (int64_t)(s >= P ? s - P : s / k) * H;
        },
        H, threadIdx.x, kSmallWaves * kWave, [&] {
          if (wave < batches) w.load(row, row_scales, wave * kBatchCols, H);
        });
    lds_sync();
    f32x4_t acc = {};
    for (int b = wave; b < batches; b += kSmallWaves) {
      if (b > wave) w.load(row, row_scales, b * kBatchCols, H);
      acc = mul_batch(w, im, b * kBatchCols, acc);
    }
    s_sum[wave][lane] = acc;
    __syncthreads();
    if (tok < m) {
      // operand row c of token t lies in lane 16 * (c / 4) + t, register c % 4
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int o = 0; o < kSmallWaves; ++o) {
        g += s_sum[o][(col / 4) * 16 + tok][col % 4];
        u += s_sum[o][((col + kUpCols) / 4) * 16 + tok][col % 4];
      }
      act[(int64_t)slot_of(s0 + tok) * I + n0 + col] = i8_swiglu(g, u);
    }
  }
}

// Down and the weighted sum: a workgroup per (token, 16 output columns), a wave per slot (in turn).
__global__ void mx4_slots_down_kernel(Mx4Experts L, int T, int k, const int32_t* __restrict__ ids,
                                      const float* __restrict__ weights, int shared, const float* __restrict__ act,
                                      void* __restrict__ Y, int out_bf16) {
  extern __shared__ __align__(16) uint8_t s_dyn[];  // [waves] images of one row, then [slots][16] parts
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int H = L.hidden, I = L.inter, P = T * k, slots = k + shared;
  const int t = blockIdx.y;
  const int n0 = blockIdx.x * 16;
  const int Kpad = (I + kBatchCols - 1) / kBatchCols * kBatchCols;
  const int each = Kpad / 2 + Kpad / kMxBlock;
  const Image im(s_dyn + (size_t)wave * each, 1, Kpad);
  float* s_part = reinterpret_cast<float*>(s_dyn + (size_t)waves * each);
  const int a = lane & 15;
  for (int s = wave; s < slots; s += waves) {
    const bool sh = s >= k;
    const int e = sh ? 0 : ids[t * k + s];
    const bool there = e >= 0 && e < L.n_experts;
    f32x4_t acc = {};
    float f = 1.0f;
    if (there) {
      const Mx4Mat down = sh ? L.sh_down : L.down;
      const int64_t r = (int64_t)e * H + n0 + a;
      const uint8_t* row = down.codes + r * (I / 2);
      const uint8_t* row_scales = down.scales + r * (I / kMxBlock);
      const int64_t slot = sh ? P + t : t * k + s;
      WeightBatch w;
      fill_image<float>(im, [&](int) { return act + slot * I; }, I, lane, kWave, [&] {
        w.load(row, row_scales, 0, I);
        if (!sh) f = weights[t * k + s];
      });
      __builtin_amdgcn_wave_barrier();
      for (int c = 0; c < I; c += kBatchCols) {
        if (c > 0) w.load(row, row_scales, c, I);
        acc = mul_batch(w, im, c, acc);
      }
      __builtin_amdgcn_wave_barrier();  // the image is read before the next slot's replaces it
    }
    if (a == 0)
      *reinterpret_cast<float4*>(s_part + s * 16 + (lane >> 4) * 4) =
          there ? make_float4(acc[0] * f, acc[1] * f, acc[2] * f, acc[3] * f) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    float y = 0.f;
    for (int s = 0; s < slots; ++s) y += s_part[s * 16 + threadIdx.x];
    const int64_t at = (int64_t)t * H + n0 + threadIdx.x;
    if (out_bf16) static_cast<uint16_t*>(Y)[at] = i8_bf16(y);
    else static_cast<float*>(Y)[at] = y;
  }
}

int down_waves(int I, int slots) {
  return std::max(1, std::min({slots, 16, (int)(kSmallLds / image_bytes(1, I))}));
}

}  // namespace

// Up to 32 tokens and 96 slots, or 128 of 256 experts and more, where fewer share an expert:
// the down product reads an expert's weights once a token, the tiles read them once.  What decides
// is the slots an expert and its size, which the rule knows only by the number of experts; whole calls
// in a graph against the tiles, us:
//   hidden 2048, intermediate 512, top-k 8 and a shared expert:
//   experts     1 token     8        12       16       20       24
//   512                  31  56   44  67   55  70            83  89
//   256         9.6 31   31  50   43  60   53  63   66  69   78  82
//   128                  30  43   41  56   52  58
//   64                   29  41   38  43   46  44
//   16                   24  34   32  34   41  35
//   hidden 4096, intermediate 1536, top-k 8, 256 experts: 8 tokens 120 141, 12 176 207, 16 223 226; 128
//   experts: 8 tokens 118 137, 12 157 152, 16 212 211; 8 experts, top-k 2: 2048 x 512 16 tokens 12 28,
//   32 tokens 17 28; 4096 x 14336 1 token 54 139, 4 tokens 100 154, 8 tokens 207 183, 32 tokens 537 185.
// So it leaves a tenth of the time to 20 and 24 tokens of 256 experts (more slots than kMaxSlots; the
// figures are with 256) and to 16 of 128, and few large experts go the slower way from 8 tokens on.
bool mx4_few_slots(const Mx4Experts& L, int64_t T, int k) {
  if (T > 32 || T * k > (L.n_experts >= 256 ? kMaxSlots : 96)) return false;
  return image_bytes(T * k < 16 ? T * k : 16, L.hidden) <= kSmallLds;
}

size_t mx4_few_slots_bytes(const Mx4Experts& L, int64_t T, int k) {
  return (size_t)(T * k + (L.sh_gate.codes ? T : 0)) * L.inter * 4;
}

hipError_t run_mx4_few_slots(const Mx4Experts& L, const uint16_t* X, int T, const int32_t* ids, const float* weights,
                             int k, void* Y, int out_bf16, float* act, hipStream_t stream) {
  const int shared = L.sh_gate.codes ? 1 : 0, P = T * k;
  const int m = std::min(std::max(P, T), 16);
  hipLaunchKernelGGL(mx4_slots_up_kernel, dim3(L.inter / kUpCols, P + shared), dim3(kSmallWaves * kWave),
                     image_bytes(m, L.hidden), stream, L, X, T, k, ids, act);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int waves = down_waves(L.inter, k + shared);
  const size_t lds = (size_t)waves * image_bytes(1, L.inter) + (size_t)(k + shared) * 64;
  hipLaunchKernelGGL(mx4_slots_down_kernel, dim3(L.hidden / 16, T), dim3(waves * kWave), lds, stream, L, T, k, ids,
                     weights, shared, act, Y, out_bf16);
  return hipGetLastError();
}

}  // namespace q4moe
