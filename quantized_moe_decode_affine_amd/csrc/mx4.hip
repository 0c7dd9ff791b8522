// Microscaled 4-bit floating point: quantization of rows, values from codes, the dense
// product Y = Xq Wq^T (mx4_gemm) and the experts' feed-forward on such products from given
// expert ids and weights (moe_experts_mx4).
//
// A product of two elements times the two blocks' scales is exact in fp32; the matrix
// instructions (v_mfma_scale_f32_32x32x64_f8f6f4 on 4-bit operands) take the scales of 32
// columns per operand row as exponent bytes and add to fp32 sums, so nothing is scaled
// outside of them.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "i8_tiles.h"
#include "steps.h"
#include "mx4.h"

namespace q4moe {

namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Rows lie end to end in values, codes and scales, so blocks are numbered through all rows.
// A lane takes half a block, the next lane the other half, so that a block's largest value is
// one exchange away and a wave reads 2 KB of consecutive bytes.  Bound by memory: 16384 x 2048 in
// 13-15 us, 5.6-6.5 TB/s (84 MB, partly held by the last cache).
constexpr int kQuantUnroll = 2;

__global__ __launch_bounds__(256) void mx4_quantize_kernel(const uint16_t* __restrict__ X, int64_t halves,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  // an even number of halves and of threads: both lanes of a block are there or neither
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < halves; i += stride * kQuantUnroll) {
    Mx4Half<uint16_t> v[kQuantUnroll];
#pragma unroll
    for (int j = 0; j < kQuantUnroll; ++j) v[j].load(X + min(i + j * stride, halves - 2 + (i & 1)) * 16);
#pragma unroll
    for (int j = 0; j < kQuantUnroll; ++j) {
      const int64_t at = i + j * stride;
      if (at >= halves) break;
      uint32_t byte;
      const uint2 c = v[j].codes(&byte);
      *reinterpret_cast<uint2*>(codes + at * 8) = c;
      if ((at & 1) == 0) scales[at >> 1] = (uint8_t)byte;
    }
  }
}

// Eight codes a lane.  e2m1 times a power of two is exact in bf16, down to its subnormals; a
// magnitude of 2^128 and more becomes infinite.  Bound by memory: 16384 x 2048 in 17-18 us.
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t eighths,
                                                             uint16_t* __restrict__ Y) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < eighths; i += stride) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + i * 4), byte = scales[i >> 2];
    const float s = byte == 255u ? __uint_as_float(0x7FC00000u) : mx4_scale(byte);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = (c >> (4 * j)) & 7u;
      // 0.5 m below 1; above, exponent m / 2 and the half of an odd code
      const float a = m < 2u ? 0.5f * (float)m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
      o[j] = (__float_as_uint(a * s) >> 16) | ((c >> (4 * j + 3)) & 1u) << 15;
    }
    uint4 v;
    v.x = o[0] | o[1] << 16;
    v.y = o[2] | o[3] << 16;
    v.z = o[4] | o[5] << 16;
    v.w = o[6] | o[7] << 16;
    *reinterpret_cast<uint4*>(Y + i * 8) = v;
  }
}

// ---- tiled product on the 4-bit matrix cores
enum { kEpiF32 = 0, kEpiBf16 = 1, kEpiSwiglu = 2, kEpiPart = 3 };

struct Mx4GemmArgs {
  const uint8_t* A;        // codes of the rows [.][K/2]
  const uint8_t* sa;       // their scales [.][K/32]
  const int32_t* row_src;  // grouped: row of A of each sorted position (null: the position itself)
  const int4* tiles;       // grouped: {expert (-1 shared, -2 none), first position, rows, 0}; null: dense
  int64_t rows;            // dense: rows of A
  uint32_t a_rows;         // gathered: rows of A (a_rows * K/2 at most 2^32 - 2^20)
  int64_t P;               // grouped: routed positions; position P + t is token t's for the shared expert
  int K, N;                // N output columns (SwiGLU: gate columns, as many up columns)
  Mx4Mat W, W2;            // weights (stacked by expert), SwiGLU: gate and up
  Mx4Mat S, S2;            // the shared expert's
  int n_slices;            // column slices of a tile
  int64_t tiles_n;         // row tiles
  void* out;               // [position][N]; SwiGLU: codes [position][N/2]
  uint8_t* out_scales;     // SwiGLU: [position][N/32]
};

constexpr int kStepBytes = 128;  // bytes of a K step, one cache line of every operand row: 256 columns
constexpr int kStepScales = kStepBytes * 2 / kMxBlock;  // and its 8 scales a row
constexpr int kBand = 4;  // tile rows of a band: the 32 workgroups of an XCD at a time cover 4 x 8 tiles (8: the same)

__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }

template <typename F, int... St>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, St...>) {
  (f(std::integral_constant<int, St>{}), ...);
}

constexpr int lcm(int a, int b) { return a % b == 0 ? a : b % a == 0 ? b : a * b; }

// Workgroup = WM x WN waves, each FM x FN blocks of 32 x 32.  Codes: each 256-column K step of
// both operands goes through LDS by 16-byte DMA loads (8 lanes read a row's whole line) in
// kStages stages, the eight 16-byte pieces of a row XOR-rotated by row bits 1-3 so that the
// operand reads (a row per lane) spread over all banks.  Scales: 8 bytes a row and K step are
// too short a piece for such loads, so a thread holds one row's scales of two K steps, loaded
// while the ones before are multiplied, and puts them into the other of two LDS buffers at the
// end; a lane then reads its row's 8 bytes once a K step and keeps the 4 that its half of the
// wave multiplies with.  K is a multiple of 64; the last K step is filled up with zeros.
// Where rows of scales are 16-byte aligned (kWide) DMA brings 64 bytes of each at a time
// instead: 8192 x 8192 x 4096 with the rows' quantization 173 us against 185.
//
// The tiles alone take 150 us of that, 3.7 PFLOP/s; the matrix instructions alone, on such data,
// reach 6.2.  Bound by the LDS reads and the matrix instructions of the two waves of a SIMD, which
// overlap in part: of the 185 us with a thread's scales 163 were left without the loads and 111
// without the multiplications.  Beside those 185, four waves of 128 x 128 instead of eight read less
// from LDS, but hide less (192-199 us); raising a wave's priority around its multiplications changed
// nothing.
template <int WM, int WN, int FM, int FN, int kStages, int EPI, bool kWide>
__device__ __forceinline__ void mx4_tile_body(const Mx4GemmArgs& p) {
  constexpr int TM = WM * FM * 32, TN = WN * FN * 32, kWaves = WM * WN;
  constexpr int kOps = (TM + TN) / 8 / kWaves;  // DMA loads per wave and step, 8 rows each
  static_assert((TM + TN) / 8 % kWaves == 0 && (kStages == 2 || kStages == 3), "whole blocks of 8 rows per wave");
  static_assert(TM + TN <= kWaves * kWave, "a thread for each row's scales");
  constexpr int kStageBytes = (TM + TN) * kStepBytes;
  // Wide: one buffer of kScale K steps, 64 bytes a row, or 32 where three stages leave no room for more.
  // Otherwise two of two K steps; a row's 16 bytes padded to 24 spread 32 rows over all banks, unpadded
  // two rows share a bank.
  constexpr int kScale = !kWide ? 2 : kStages == 2 ? 8 : 4;
  constexpr int kScalePitch = kScale * kStepScales + (!kWide && kStages == 2 ? 8 : 0);
  // one array per stage, so that the compiler can tell a stage's reads from the loads
  // still filling another
  __shared__ __align__(16) uint8_t s_st0[kStageBytes], s_st1[kStageBytes];
  uint8_t* st2 = nullptr;
  if constexpr (kStages > 2) {
    __shared__ __align__(16) uint8_t s_st2[kStageBytes];
    st2 = s_st2;
  }
  __shared__ __align__(16) uint8_t s_sc[kWide ? 1 : 2][(TM + TN) * kScalePitch];
  constexpr bool kSwiglu = EPI == kEpiSwiglu;
  constexpr int kCols = kSwiglu ? TN / 2 : TN;  // output columns of a tile
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int Kb = p.K / 2, Ks = p.K / kMxBlock;

  // Workgroups go to the XCDs in turn.  Grouped: all slices of a tile stay on one (they read
  // the same rows of A).  Dense: an XCD takes a run of the tiles in bands of kBand tile rows,
  // so that the workgroups it runs at a time share rows of A and of W in its L2.
  const uint32_t xcd = blockIdx.x % kXcds, q = blockIdx.x / kXcds, slices = p.n_slices;
  uint32_t tile, slice;
  if (p.tiles) {
    tile = q / slices * kXcds + xcd;
    slice = q % slices;
  } else {
    const uint32_t id = xcd * (gridDim.x / kXcds) + q;
    if (id >= (uint32_t)p.tiles_n * slices) return;  // the grid is rounded up to the XCDs
    const uint32_t band = id / (kBand * slices), in_band = id - band * (kBand * slices);
    const uint32_t high = min((uint32_t)kBand, (uint32_t)p.tiles_n - band * kBand);
    tile = band * kBand + in_band % high;
    slice = in_band / high;
  }
  // (uniform, but divisions leave them in vector registers)
  tile = __builtin_amdgcn_readfirstlane(tile);
  slice = __builtin_amdgcn_readfirstlane(slice);
  if (tile >= p.tiles_n) return;
  const int n0 = (int)slice * kCols;
  int expert = 0;
  int64_t first = (int64_t)tile * TM;
  int rows;
  if (p.tiles) {
    const int4 tl = p.tiles[tile];
    expert = __builtin_amdgcn_readfirstlane(tl.x);
    if (expert == -2) return;
    first = __builtin_amdgcn_readfirstlane(tl.y);
    rows = __builtin_amdgcn_readfirstlane(tl.z);
  } else {
    rows = min(TM, (int)min(p.rows - first, (int64_t)TM));
  }
  const Mx4Mat w = expert < 0 ? p.S : p.W, w2 = expert < 0 ? p.S2 : p.W2;
  const int64_t e_row = (int64_t)max(expert, 0) * p.N;  // first row of this expert's matrix
  auto source = [&](int r) -> int64_t {  // row of A of the tile's row r
    const int64_t pos = first + min(r, rows - 1);
    return !p.row_src ? pos : pos < p.P ? (int64_t)p.row_src[pos] : pos - p.P;
  };

  // Loads of this wave: kOpsA blocks of 8 rows of A and kOpsW of W.  The buffers' bounds are
  // the matrix (or the tile's rows): what lies beyond reads as zero, and the 32-bit offsets
  // need no arithmetic per step.  SwiGLU: the first half of the loads are gate rows, the
  // second the up rows of the same columns, placed so that a wave's first FN/2 blocks of 32
  // columns are gate and the rest up, and a lane holds both.
  constexpr int kOpsA = TM / 8 / kWaves, kOpsW = TN / 8 / kWaves;
  constexpr int kOpsG = kSwiglu ? kOpsW / 2 : kOpsW;
  constexpr int kPairs = FN > 1 ? FN / 2 : 1;  // SwiGLU: a wave's gate blocks, and its up blocks
  static_assert(!kSwiglu || FN % 2 == 0, "gate and up blocks come in pairs");
  int off[kOps], dst[kOps];
  const int piece = lane & 7;
#pragma unroll
  for (int j = 0; j < kOps; ++j) {
    int blk;  // block of 8 rows in the stage
    uint32_t row;  // row of the operand
    bool inside = true;
    if (j < kOpsA) {
      blk = wave * kOpsA + j;
      const int r = blk * 8 + (lane >> 3);
      row = p.row_src ? (uint32_t)source(r) : (uint32_t)r;  // gathered rows: offsets from the whole matrix
      inside = r < rows;
    } else {
      const bool up = j - kOpsA >= kOpsG;
      const int i = wave * kOpsG + (j - kOpsA) % kOpsG;  // block of 8 of this matrix's columns
      row = i * 8 + (lane >> 3);
      const int b = i / 4;  // block of 32 of them
      blk = TM / 8 + (kSwiglu ? (b / kPairs * FN + b % kPairs + (up ? kPairs : 0)) * 4 + i % 4 : i);
    }
    const int r = blk * 8 + (lane >> 3);
    // a row past the tile's last one lies beyond every buffer: it costs no traffic
    off[j] = inside ? (int)(row * (uint32_t)Kb + (uint32_t)(piece ^ row_swz(r)) * 16) : (int)0xFFFFFFF0u;
    dst[j] = blk * 8 * kStepBytes;
  }
  auto rsrc = [&](const uint8_t* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)bytes, kBufferRsrcWord3);
  };
  const int64_t w_off = (e_row + n0) * Kb;
  const uint32_t w_bytes = (uint32_t)min(kCols, p.N - n0) * (uint32_t)Kb;  // a tile's rows: at most 256 * 32768
  const __amdgpu_buffer_rsrc_t ra =
      rsrc(p.row_src ? p.A : p.A + first * Kb, (p.row_src ? p.a_rows : (uint32_t)rows) * (uint32_t)Kb);
  const __amdgpu_buffer_rsrc_t rw = rsrc(w.codes + w_off, w_bytes), ru = rsrc(w2.codes + w_off, w_bytes);
  auto stage = [&](int st) -> uint8_t* { return st == 0 ? s_st0 : st == 1 ? s_st1 : st2; };
  const int steps = (Kb + kStepBytes - 1) / kStepBytes;
  // Steps past the last load it again and are not computed.  Of the last step what lies past
  // a row's end is zeros on A's side (loads beyond the buffer), so whatever W's side has there
  // adds nothing.
  auto issue_op = [&](int i, int st, int j) __attribute__((always_inline)) {
    const int k0 = min(i, steps - 1) * kStepBytes;
    const __amdgpu_buffer_rsrc_t r = j < kOpsA ? ra : j < kOpsA + kOpsG ? rw : ru;
    int at = off[j];
    if (j < kOpsA && k0 + (piece ^ row_swz((wave * kOpsA + j) * 8 + (lane >> 3))) * 16 >= Kb) at = (int)0xFFFFFFF0u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, stage(st) + dst[j], 16, at, k0, 0, 0);
  };

  // ---- scales, narrow: this thread's row (threads beyond the rows repeat some).  Rows and columns
  // outside the matrices take another's: their sums are not stored.
  const int srow = threadIdx.x % (TM + TN);
  const uint8_t* sp = p.sa;
  if (kWide) {
  } else if (srow < TM) {
    sp = p.sa + source(srow) * Ks;
  } else {
    const int b = (srow - TM) / 32;  // block of 32 rows of the stage
    const bool up = kSwiglu && b % FN >= kPairs;
    const int col = (kSwiglu ? b / FN * kPairs + b % kPairs : b) * 32 + srow % 32;
    sp = (up ? w2.scales : w.scales) + (e_row + min(n0 + col, p.N - 1)) * Ks;
  }
  // Without a branch, which would let the compiler move products over the barriers: a K step's
  // 8 bytes, for a row's last ones those that end with it, shifted, with zeros (2^-127) behind;
  // steps past the last are not used.
  uint64_t held[kScale];
  auto load_scales = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < kScale; ++o) {
      const int at = (chunk * kScale + o) * kStepScales, from = min(at, max(Ks, kStepScales) - kStepScales);
      __builtin_memcpy(&held[o], sp + from, kStepScales);
    }
  };
  auto load_short = [&] {  // rows of fewer than 8: one K step
    held[0] = 0;
#pragma unroll
    for (int o = 0; o < kStepScales / 2; ++o)
      held[0] |= (uint64_t)*reinterpret_cast<const uint16_t*>(sp + min(2 * o, Ks - 2)) << (16 * o);
#pragma unroll
    for (int o = 1; o < kScale; ++o) held[o] = 0;
    sp = p.A;  // what is loaded from here on is not used: 8 bytes that are there
  };
  auto scale_at = [&](int r, int step) { return r * kScalePitch + step * kStepScales; };
  auto put_scales = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < kScale; ++o) {
      const int at = (chunk * kScale + o) * kStepScales, from = min(at, max(Ks, kStepScales) - kStepScales);
      // (shifted here, not where it is loaded: a use would wait for the load)
      *reinterpret_cast<uint64_t*>(s_sc[chunk & 1] + scale_at(srow, o)) = held[o] >> min(at - from, kStepScales - 1) * 8;
    }
  };

  // ---- scales, wide: DMA loads of 16 bytes, kPieces lanes to a row.  A row's pieces are XOR-rotated by the
  // rows whose banks would repeat.
  constexpr int kPieces = kScale * kStepScales / 16, kRowsPer = kWave / kPieces;
  constexpr int kScaleOps = ((TM + TN) / kRowsPer + kWaves - 1) / kWaves;  // loads per wave and buffer
  auto piece_swz = [](int r) { return kPieces == 4 ? (r >> 2) & 3 : (r >> 3) & 1; };
  int soff[kWide ? kScaleOps : 1];
  // (uniform) first row of the j-th load's rows in the stage; the last ones repeat some
  auto scale_rows = [&](int j) { return min(wave * kScaleOps + j, (TM + TN) / kRowsPer - 1) * kRowsPer; };
  if constexpr (kWide) {
#pragma unroll
    for (int j = 0; j < kScaleOps; ++j) {
      const int r = scale_rows(j) + lane / kPieces;
      uint32_t row;
      bool inside = true;
      if (r < TM) {
        row = p.row_src ? (uint32_t)source(r) : (uint32_t)r;
        inside = r < rows;
      } else {
        const int blk = (r - TM) / 32;
        row = (kSwiglu ? blk / FN * kPairs + blk % kPairs : blk) * 32 + r % 32;
      }
      soff[j] = inside ? (int)(row * (uint32_t)Ks + (uint32_t)(lane % kPieces ^ piece_swz(r)) * 16) : (int)0xFFFFFFF0u;
    }
  }
  // (the chunk after the last one is not used: it repeats the last)
  auto issue_scales = [&](int chunk) __attribute__((always_inline)) {
    const int k0 = min(chunk, (steps - 1) / kScale) * (kScale * kStepScales);
#pragma unroll
    for (int j = 0; j < kScaleOps; ++j) {
      // which matrix: uniform, and selected as an address (a selected descriptor went through scratch memory)
      const int r = scale_rows(j);
      const uint8_t* at = p.row_src ? p.sa : p.sa + first * Ks;
      uint32_t bytes = (p.row_src ? p.a_rows : (uint32_t)rows) * (uint32_t)Ks;
      if (r >= TM) {
        at = (kSwiglu && (r - TM) / 32 % FN >= kPairs ? w2.scales : w.scales) + (e_row + n0) * Ks;
        bytes = (uint32_t)min(kCols, p.N - n0) * (uint32_t)Ks;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(at, bytes), s_sc[0] + r * kScalePitch, 16, soff[j], k0, 0, 0);
    }
  };

  // Operand reads run one MFMA step (64 columns) ahead of the products.  At the end of a K
  // step, with the last 64 columns' operands in registers, the workgroup meets: every wave
  // has read the stage, so its next loads go out, the next stage's first operands are read,
  // and the last products cover both.
  const int m = lane & 31, h = lane >> 5;
  const uint32_t pick = h ? 0x07050301u : 0x06040200u;  // of a row's 8 scales those of blocks 2 kk + h
  f32x16_t acc[FM][FN] = {};
  auto run = [&](auto nf_c) __attribute__((always_inline)) {
    constexpr int NF = decltype(nf_c)::value;
    i32x4_t a[2][NF > 0 ? NF : 1], b[2][FN];
    uint32_t xa[NF > 0 ? NF : 1], xb[FN];
    auto read = [&](const uint8_t* base, int kk, int set) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);  // these reads go out before the products that follow in the source
      if constexpr (NF > 0) {
        // (a row's rotation is that of the row 32 further: one address for all blocks)
        const int c = ((2 * kk + h) ^ row_swz(m)) << 4;
#pragma unroll
        for (int f = 0; f < NF; ++f)
          a[set][f] = *reinterpret_cast<const i32x4_t*>(base + (wm * FM * 32 + m) * kStepBytes + c + f * 32 * kStepBytes);
#pragma unroll
        for (int f = 0; f < FN; ++f)
          b[set][f] = *reinterpret_cast<const i32x4_t*>(base + (TM + wn * FN * 32 + m) * kStepBytes + c + f * 32 * kStepBytes);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // a K step's scales: a row's eight, on their way while the last products of the step before run,
    // then those of them that this lane multiplies with
    typedef typename std::conditional<kWide, uint4, uint2>::type raw_t;  // wide: of two K steps
    raw_t raw_a[NF > 0 ? NF : 1], raw_b[FN];
    auto read_scales = [&](int buffer, int step) __attribute__((always_inline)) {
      if constexpr (NF > 0) {
        const int in_row = kWide ? (step / 2 ^ piece_swz(m)) * 16 : step * kStepScales;  // (as that of the row 32 further)
        const uint8_t* at = s_sc[kWide ? 0 : buffer] + in_row;
#pragma unroll
        for (int f = 0; f < NF; ++f)
          raw_a[f] = *reinterpret_cast<const raw_t*>(at + (wm * FM * 32 + m) * kScalePitch + f * 32 * kScalePitch);
#pragma unroll
        for (int f = 0; f < FN; ++f)
          raw_b[f] = *reinterpret_cast<const raw_t*>(at + (TM + wn * FN * 32 + m) * kScalePitch + f * 32 * kScalePitch);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto take_scales = [&](auto u_c) __attribute__((always_inline)) {
      auto mine = [&](const auto& v) {
        if constexpr (kWide && decltype(u_c)::value % 2 == 1) return __builtin_amdgcn_perm(v.w, v.z, pick);
        else return __builtin_amdgcn_perm(v.y, v.x, pick);
      };
      if constexpr (NF > 0) {
#pragma unroll
        for (int f = 0; f < NF; ++f) xa[f] = mine(raw_a[f]);
#pragma unroll
        for (int f = 0; f < FN; ++f) xb[f] = mine(raw_b[f]);
      }
    };
    // One MFMA step of operand set kk % 2, with the loads [j0, j1) of a K step into stage st
    // between its products.
    auto mul = [&](auto kk_c, int i, auto st_c, auto j0_c, auto j1_c) __attribute__((always_inline)) {
      constexpr int kk = decltype(kk_c)::value, set = kk % 2;
      constexpr int st = decltype(st_c)::value, j0 = decltype(j0_c)::value, j1 = decltype(j1_c)::value;
      constexpr int kPer = (j1 - j0 + NF - 1) / (NF > 0 ? NF : 1);  // loads after each row of products
#pragma unroll
      for (int fm = 0; fm < NF; ++fm) {
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
          acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              mx4_operand(b[set][fn]), mx4_operand(a[set][fm]), acc[fm][fn], kFp4, kFp4, kk, (int)xb[fn], kk, (int)xa[fm]);
        if constexpr (j1 > j0) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = j0 + fm * kPer; j < min(j1, j0 + (fm + 1) * kPer); ++j) issue_op(i, st, j);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (NF == 0) {
#pragma unroll
        for (int j = j0; j < j1; ++j) issue_op(i, st, j);
      }
    };
    auto meet = [&](auto left_c) __attribute__((always_inline)) {  // with that many loads in flight
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(decltype(left_c)::value));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    using C3 = std::integral_constant<int, 3>;
    using Half = std::integral_constant<int, kOps / 2>;
    using All = std::integral_constant<int, kOps>;
    // K step i = u modulo the unrolled steps.  kk = 0's operands are in set 0 and the step's
    // scales on their way on entry, and the next step's on return.
    constexpr int kUnroll = lcm(kStages, kScale);
    auto step = [&](int i, auto u_c) __attribute__((always_inline)) {
      constexpr int u = decltype(u_c)::value, st = u % kStages;
      using St = std::integral_constant<int, st>;
      using Free = std::integral_constant<int, (st + kStages - 1) % kStages>;  // the stage read before this one
      // Wide: the scales of the buffer's last two K steps were read before the workgroup last met, so its next
      // ones go out in the last of them, and land before the workgroup meets again.
      constexpr bool kNext = kWide && u % kScale == kScale - 1;
      take_scales(u_c);
      if constexpr (kNext) issue_scales(i / kScale + 1);
      if constexpr (!kWide && u % kScale == 0) load_scales(i / kScale + 1);
      read(stage(st), 1, 1);
      mul(C0{}, i + kStages - 1, Free{}, Half{}, All{});
      read(stage(st), 2, 0);
      mul(C1{}, 0, St{}, C0{}, C0{});
      read(stage(st), 3, 1);
      mul(C2{}, 0, St{}, C0{}, C0{});
      if constexpr (!kWide && u % kScale == kScale - 1) put_scales(i / kScale + 1);
      // (three stages: of what may still be in flight only the second half of this step's loads is younger)
      meet(std::integral_constant<int, (kNext && kStages > 2 ? kOps - kOps / 2 : kOps * (kStages - 2))>{});
      read(stage((st + 1) % kStages), 0, 0);
      if constexpr (!kWide || u % 2 == 1) read_scales((i + 1) / kScale & 1, (u + 1) % kScale);
      mul(C3{}, i + kStages, St{}, C0{}, Half{});
    };
    if constexpr (!kWide) {
      if (Ks < kStepScales) load_short();
      else load_scales(0);
      put_scales(0);
    }
    meet(std::integral_constant<int, kOps * (kStages - 2) + kOps / 2>{});
    read(stage(0), 0, 0);
    read_scales(0, 0);
    int i = 0;
    for (; i + kUnroll <= steps; i += kUnroll)
      each_of([&](auto u_c) { step(i + decltype(u_c)::value, u_c); }, std::make_integer_sequence<int, kUnroll>{});
    each_of(
        [&](auto u_c) {
          if (i + decltype(u_c)::value < steps) step(i + decltype(u_c)::value, u_c);
        },
        std::make_integer_sequence<int, kUnroll - 1>{});
  };
  if constexpr (kWide) issue_scales(0);
#pragma unroll
  for (int st = 0; st < kStages; ++st)
#pragma unroll
    for (int j = 0; j < (st + 1 < kStages ? kOps : kOps / 2); ++j) issue_op(st, st, j);
  // grouped tiles are often part full: only the 32-row blocks that hold rows are multiplied
  if constexpr (EPI == kEpiF32 || EPI == kEpiBf16) {
    run(std::integral_constant<int, FM>{});
  } else {
    static_assert(FM == 2, "none, one or both of a wave's blocks");
    const int has = rows - wm * FM * 32;
    if (has > 32) run(std::integral_constant<int, 2>{});
    else if (has > 0) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
  }
  __builtin_amdgcn_s_waitcnt(0);  // the repeated loads of the last steps are still landing

  if constexpr (kSwiglu) {
    // A lane holds 16 of its row's 32 activations of a block (columns 8 q + 4 h + j), the lane
    // 32 further the others: the block's codes and scale are made here, from fp32.
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int r = (wm * FM + fm) * 32 + m;
      if (r - m >= rows) break;
#pragma unroll
      for (int fn = 0; fn < FN / 2; ++fn) {
        const int c0 = n0 + (wn * (FN / 2) + fn) * 32;
        float v[16];
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          v[j] = i8_swiglu(acc[fm][fn][j], acc[fm][fn + FN / 2][j]);
          most = max(most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        }
        uint32_t x, y;
        swap_halves32(most, x, y);
        const uint32_t byte = mx4_scale_byte(max(x, y));
        const float s = mx4_scale(byte);
        uint32_t d[2] = {};  // two column quads each, this half's 16 bits of either
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          d[o] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d[o], v[8 * o + 0], v[8 * o + 1], s, 0);
          d[o] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d[o], v[8 * o + 2], v[8 * o + 3], s, 1);
          d[o] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d[o], v[8 * o + 4], v[8 * o + 5], s, 2);
          d[o] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d[o], v[8 * o + 6], v[8 * o + 7], s, 3);
          if (byte == 255u) d[o] = 0;
        }
        // the lower lanes get both halves' first two quads, the upper ones the last two
        const auto t = __builtin_amdgcn_permlane32_swap(d[0], d[1], false, false);
        const uint2 c = make_uint2(__builtin_amdgcn_perm(t[1], t[0], 0x05040100u), __builtin_amdgcn_perm(t[1], t[0], 0x07060302u));
        if (r < rows && c0 < p.N) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (first + r) * (p.N / 2) + c0 / 2 + h * 8) = c;
          if (h == 0) p.out_scales[(first + r) * (p.N / kMxBlock) + c0 / kMxBlock] = (uint8_t)byte;
        }
      }
    }
    return;
  }

  // The weight is the first operand of the products, so that a lane holds sums of one row of
  // A (lane % 32) and four consecutive output columns (8*(i/4) + 4*(lane/32) + i%4).  Stored
  // from there a column quad of 32 rows would touch 32 cache lines, at a power-of-two
  // distance for most N; so each wave turns 32 rows at a time in LDS and stores whole rows
  // of its columns, 16 bytes a lane.
  constexpr bool kHalf = EPI == kEpiBf16;
  typedef typename std::conditional<kHalf, uint16_t, float>::type out_t;
  constexpr int kRow = FN * 32 * sizeof(out_t), kPitch = kRow + 16;  // the pad spreads the rows over the banks
  constexpr int kVec = 16 / sizeof(out_t);
  static_assert(kWaves % 2 == 0 && kWaves / 2 * 32 * kPitch <= kStageBytes, "the waves' blocks fit two stages");
  uint8_t* turn = (wave < kWaves / 2 ? s_st0 : s_st1) + wave % (kWaves / 2) * 32 * kPitch;
  const bool whole = p.N % kVec == 0;  // 16 bytes of a row are inside or outside together, and aligned
  const int c0 = n0 + wn * FN * 32;
  __builtin_amdgcn_s_barrier();  // no wave reads the stages any more
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int r0 = (wm * FM + fm) * 32;
    if (r0 >= rows) break;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint8_t* to = turn + m * kPitch + (fn * 32 + 8 * q + 4 * h) * sizeof(out_t);
        const float o[4] = {acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1], acc[fm][fn][4 * q + 2], acc[fm][fn][4 * q + 3]};
        if constexpr (kHalf)
          *reinterpret_cast<uint2*>(to) =
              make_uint2(i8_bf16(o[0]) | (uint32_t)i8_bf16(o[1]) << 16, i8_bf16(o[2]) | (uint32_t)i8_bf16(o[3]) << 16);
        else
          *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
      }
    __builtin_amdgcn_wave_barrier();  // the block is the wave's own, and LDS keeps its order
    constexpr int kLanes = kRow / 16;
#pragma unroll
    for (int b = 0; b < 32; b += kWave / kLanes) {
      const int r = b + lane / kLanes, c = lane % kLanes * kVec;
      const uint4 v = *reinterpret_cast<const uint4*>(turn + r * kPitch + c * sizeof(out_t));
      if (r0 + r >= rows || c0 + c >= p.N) continue;
      out_t* out = static_cast<out_t*>(p.out) + (first + r0 + r) * p.N + c0 + c;
      if (whole) {
        *reinterpret_cast<uint4*>(out) = v;
      } else {
        out_t e[kVec];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (c0 + c + j < p.N) out[j] = e[j];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int WM, int WN, int FM, int FN, int kStages, int EPI, bool kWide>
__global__ __launch_bounds__(WM* WN* kWave, 2) void mx4_tile_kernel(Mx4GemmArgs p) {
  mx4_tile_body<WM, WN, FM, FN, kStages, EPI, kWide>(p);
}

// Rows of scales that 16-byte loads can take.
bool wide_scales(const Mx4GemmArgs& p) {
  uintptr_t at = reinterpret_cast<uintptr_t>(p.sa) | (uintptr_t)(p.K / kMxBlock);
  for (const Mx4Mat* m : {&p.W, &p.W2, &p.S, &p.S2}) at |= reinterpret_cast<uintptr_t>(m->scales);
  return at % 16 == 0;
}

template <int WM, int WN, int FM, int FN, int kStages, int EPI>
hipError_t launch_tiles(Mx4GemmArgs p, int64_t tiles, hipStream_t stream) {
  constexpr int kCols = WN * FN * 32 / (EPI == kEpiSwiglu ? 2 : 1);
  p.n_slices = (p.N + kCols - 1) / kCols;
  p.tiles_n = tiles;
  const int64_t blocks = p.tiles ? (tiles + kXcds - 1) / kXcds * kXcds * p.n_slices
                                 : (tiles * p.n_slices + kXcds - 1) / kXcds * kXcds;
  if (blocks <= 0) return hipSuccess;
  if (blocks * (WM * WN * kWave) > kMaxThreads) return hipErrorInvalidValue;  // bounded by the callers
  const dim3 grid((unsigned)blocks), threads(WM * WN * kWave);
  if (wide_scales(p)) hipLaunchKernelGGL((mx4_tile_kernel<WM, WN, FM, FN, kStages, EPI, true>), grid, threads, 0, stream, p);
  else hipLaunchKernelGGL((mx4_tile_kernel<WM, WN, FM, FN, kStages, EPI, false>), grid, threads, 0, stream, p);
  return hipGetLastError();
}

// y[t] = sum_i (down product of slot i) w_i + shared, in slot order, the shared expert last;
// slots whose id names no expert add nothing.  Bound by the products' bytes, written just before:
// 2048 tokens of 2048, top-k 8 and a shared expert: 28 us for 160 MB, 5.7 TB/s.
__global__ __launch_bounds__(256) void mx4_combine_kernel(const float* __restrict__ part, const int32_t* __restrict__ inv,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ weights, int64_t T, int k, int E,
                                                          int H, int64_t P, int shared, void* __restrict__ Y,
                                                          int out_bf16) {
  const int per = H / 8;
  const int64_t total = T * per;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per;
    const int n = (int)(i - t * per) * 8;
    float y[8] = {};
    auto add = [&](int64_t pos, float f) {
      const float4* q = reinterpret_cast<const float4*>(part + pos * H + n);
      const float4 a = q[0], b = q[1];
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = i8_add_slot(y[j], v[j], f);
    };
    for (int s0 = 0; s0 < k; s0 += 4) {  // four slots' loads in flight
      int64_t pos[4];
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = t * k + min(s0 + j, k - 1);
        const int e = ids[r];
        pos[j] = s0 + j < k && e >= 0 && e < E ? inv[r] : -1;
        f[j] = weights[r];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (pos[j] >= 0) add(pos[j], f[j]);
    }
    if (shared) add(P + t, 1.0f);
    if (out_bf16) {
      uint4 o;
      o.x = (uint32_t)i8_bf16(y[0]) | ((uint32_t)i8_bf16(y[1]) << 16);
      o.y = (uint32_t)i8_bf16(y[2]) | ((uint32_t)i8_bf16(y[3]) << 16);
      o.z = (uint32_t)i8_bf16(y[4]) | ((uint32_t)i8_bf16(y[5]) << 16);
      o.w = (uint32_t)i8_bf16(y[6]) | ((uint32_t)i8_bf16(y[7]) << 16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(Y) + t * H + n) = o;
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(Y) + t * H + n);
      o[0] = make_float4(y[0], y[1], y[2], y[3]);
      o[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
}

// Rows of a grouped tile: 128 x 256 columns by eight waves.  2048 tokens, top-k 8 of 256
// experts, hidden 2048, intermediate 512: quantization 5 us, sorting 12, gate and up 86, down 72,
// combining 28 (kernel times).  64 rows an expert on average leave half of a tile's rows empty, and each
// tile reads its weights once, 429 MB in all at 2.7 TB/s: bound by the tiles' latency, as gate and up have
// 8 K steps and the down product 2.
// Tiles of 128 x 128, two to a compute unit: 205 us against 203; 512 tokens 145 against 150.
constexpr int kExpertRows = 128;

struct ExpertsWs {
  uint8_t *xq, *sx;      // [T][H/2] codes of the tokens, [T][H/32] scales
  int32_t *offsets, *sorted, *inv, *row_src;
  float* row_w;
  int4* tiles;
  void* perm;
  uint8_t *aq, *sh;      // [R][I/2], [R][I/32] silu(gate) * up of each sorted position
  float* part;           // [R][H] the down product
  size_t total;
};

ExpertsWs carve(void* base, const Mx4Experts& L, int64_t T, int k) {
  ExpertsWs w{};
  char* c = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) { char* r = c ? c + off : nullptr; off += align256(bytes); return r; };
  const int64_t P = T * k, extra = L.sh_gate.codes ? T : 0, R = P + extra;
  w.xq = reinterpret_cast<uint8_t*>(take((size_t)T * L.hidden / 2));
  w.sx = reinterpret_cast<uint8_t*>(take((size_t)T * L.hidden / kMxBlock));
  w.offsets = reinterpret_cast<int32_t*>(take((size_t)(L.n_experts + 1) * 4));
  w.sorted = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  w.inv = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  w.row_src = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  w.row_w = reinterpret_cast<float*>(take((size_t)P * 4));
  w.tiles = reinterpret_cast<int4*>(take((size_t)group_max_tiles(P, L.n_experts, extra, kExpertRows) * 16));
  w.perm = take(permute_workspace_bytes(P, L.n_experts));
  w.aq = reinterpret_cast<uint8_t*>(take((size_t)R * L.inter / 2));
  w.sh = reinterpret_cast<uint8_t*>(take((size_t)R * L.inter / kMxBlock));
  w.part = reinterpret_cast<float*>(take((size_t)R * L.hidden * 4));
  w.total = off;
  return w;
}

}  // namespace

hipError_t run_mx4_quantize(const uint16_t* X, int64_t rows, int K, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t halves = rows * (K / 16);
  if (halves <= 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((halves + 256 * kQuantUnroll - 1) / (256 * kQuantUnroll), 1 << 16));
  hipLaunchKernelGGL(mx4_quantize_kernel, grid, dim3(256), 0, stream, X, halves, codes, scales);
  return hipGetLastError();
}

hipError_t run_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* Y,
                              hipStream_t stream) {
  const int64_t eighths = rows * (K / 8);
  if (eighths <= 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((eighths + 255) / 256, 1 << 16));
  hipLaunchKernelGGL(mx4_dequantize_kernel, grid, dim3(256), 0, stream, codes, scales, eighths, Y);
  return hipGetLastError();
}

size_t mx4_gemm_workspace_bytes(int64_t m, int K) { return align256((size_t)m * K / 2) + align256((size_t)m * K / kMxBlock); }

hipError_t run_mx4_gemm(const Mx4Mat& W, int64_t n, int K, const uint16_t* X, int64_t m, void* Y, int out_bf16, void* ws,
                        hipStream_t stream) {
  if (mx4_few_rows(m, K)) return run_mx4_few_rows(W, n, K, X, (int)m, Y, out_bf16, stream);
  uint8_t* xq = static_cast<uint8_t*>(ws);
  uint8_t* sx = xq + align256((size_t)m * K / 2);
  const hipError_t e = run_mx4_quantize(X, m, K, xq, sx, stream);
  if (e != hipSuccess) return e;
  Mx4GemmArgs p{};
  p.A = xq;
  p.sa = sx;
  p.rows = m;
  p.K = K;
  p.N = (int)n;
  p.W = p.W2 = p.S = p.S2 = W;
  p.out = Y;
  // The 8-bit product's rule, which fits here as well (us on tiles of 256 / 128 / 64): 64 rows of
  // 2048 x 2048 18 / 13 / 10; 512 x 8192 x 4096 33 / 23 / 27; 2048 x 4096 x 4096 38 / 33 / 45;
  // 4096 x 4096 x 4096 48 / 59 / 84.
  const int tile = i8_dense_tile(m, n, device_cu_count());
  if (tile == 256)
    return out_bf16 ? launch_tiles<2, 4, 4, 2, 2, kEpiBf16>(p, (m + 255) / 256, stream)
                    : launch_tiles<2, 4, 4, 2, 2, kEpiF32>(p, (m + 255) / 256, stream);
  if (tile == 128)
    return out_bf16 ? launch_tiles<2, 2, 2, 2, 2, kEpiBf16>(p, (m + 127) / 128, stream)
                    : launch_tiles<2, 2, 2, 2, 2, kEpiF32>(p, (m + 127) / 128, stream);
  return out_bf16 ? launch_tiles<2, 2, 1, 1, 3, kEpiBf16>(p, (m + 63) / 64, stream)
                  : launch_tiles<2, 2, 1, 1, 3, kEpiF32>(p, (m + 63) / 64, stream);
}

size_t experts_mx4_workspace_bytes(const Mx4Experts& L, int64_t T, int k) {
  // a workspace made for T tokens also takes fewer, the few-slots form among them
  return std::max(carve(nullptr, L, T, k).total, align256(mx4_few_slots_bytes(L, T, k)));
}

hipError_t run_moe_experts_mx4(const Mx4Experts& L, const uint16_t* X, int64_t T, const int32_t* ids,
                               const float* weights, int k, void* Y, int out_bf16, void* ws, hipStream_t stream) {
  if (mx4_few_slots(L, T, k))
    return run_mx4_few_slots(L, X, (int)T, ids, weights, k, Y, out_bf16, static_cast<float*>(ws), stream);
  const int H = L.hidden, I = L.inter, E = L.n_experts;
  const ExpertsWs w = carve(ws, L, T, k);
  const int64_t P = T * k, extra = L.sh_gate.codes ? T : 0;
  const int max_tiles = group_max_tiles(P, E, extra, kExpertRows);
  GroupTiles gt{};
  gt.tile_rows = kExpertRows;
  gt.max_tiles = max_tiles;
  gt.extra_rows = extra;
  gt.topk = k;
  gt.table = w.tiles;
  gt.row_src = w.row_src;
  gt.row_w = w.row_w;
  hipError_t e = run_mx4_quantize(X, T, H, w.xq, w.sx, stream);
  if (e != hipSuccess) return e;
  e = run_permute(ids, P, E, w.offsets, w.sorted, w.inv, w.perm, &gt, stream);
  if (e != hipSuccess) return e;

  Mx4GemmArgs p{};
  p.A = w.xq;
  p.sa = w.sx;
  p.row_src = w.row_src;
  p.a_rows = (uint32_t)T;
  p.tiles = w.tiles;
  p.P = P;
  p.K = H;
  p.N = I;
  p.W = L.gate;
  p.W2 = L.up;
  p.S = L.sh_gate;
  p.S2 = L.sh_up;
  p.out = w.aq;
  p.out_scales = w.sh;
  e = launch_tiles<2, 4, 2, 2, 3, kEpiSwiglu>(p, max_tiles, stream);
  if (e != hipSuccess) return e;

  Mx4GemmArgs d = p;
  d.A = w.aq;
  d.sa = w.sh;
  d.row_src = nullptr;
  d.K = I;
  d.N = H;
  d.W = d.W2 = L.down;
  d.S = d.S2 = L.sh_down;
  d.out = w.part;
  e = launch_tiles<2, 4, 2, 2, 3, kEpiPart>(d, max_tiles, stream);
  if (e != hipSuccess) return e;

  const unsigned blocks = (unsigned)std::min<int64_t>((T * (H / 8) + 255) / 256, 65536);
  hipLaunchKernelGGL(mx4_combine_kernel, dim3(blocks), dim3(256), 0, stream, w.part, w.inv, ids, weights, T, k, E, H, P,
                     extra ? 1 : 0, Y, out_bf16);
  return hipGetLastError();
}

}  // namespace q4moe
