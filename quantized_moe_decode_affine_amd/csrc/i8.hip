// Products in 8-bit integers: quantization of rows, the dense product Y = X W^T with a
// scale per token and per output channel (i8_gemm), and the experts' feed-forward on such
// products from given expert ids and weights (moe_experts_i8).
//
//   Y[m][n] = (float(sum_k q[m][k] c[n][k]) * sx[m]) * sw[n]
//
// with q, sx the symmetric 8-bit rows of X (int8.h) and c, sw the weight's codes and
// channel scales.  The integer sum is exact in 32 bits (k is bounded on the host), so every
// tiling and order gives the same sums, and an output is rounded when the sum becomes a
// float, at each of the two scales and to its own type.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "i8_tiles.h"
#include "int8.h"
#include "kernels.h"

namespace q4moe {

namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// One wave per row; bound by the row's bytes: 8192 x 4096 in 26-31 us, 100 MB (3.2-3.9 TB/s).
template <typename In, int kHeld>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const In* __restrict__ X, int64_t rows, int K,
                                                          int8_t* __restrict__ codes, float* __restrict__ scales) {
  for (int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; r < rows; r += (int64_t)gridDim.x * 4)
    i8_quantize_row<kHeld>(X + r * K, K, codes + r * K, scales + r);
}

template <typename In>
hipError_t launch_quantize(const In* X, int64_t rows, int K, int8_t* codes, float* scales, hipStream_t stream) {
  if (rows <= 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((rows + 3) / 4, 1 << 20)), threads(256);
  if (K <= 512)
    hipLaunchKernelGGL((i8_quantize_kernel<In, 1>), grid, threads, 0, stream, X, rows, K, codes, scales);
  else if (K <= 2048)
    hipLaunchKernelGGL((i8_quantize_kernel<In, 4>), grid, threads, 0, stream, X, rows, K, codes, scales);
  else
    hipLaunchKernelGGL((i8_quantize_kernel<In, 8>), grid, threads, 0, stream, X, rows, K, codes, scales);
  return hipGetLastError();
}

// ---- tiled product on the i8 matrix cores
enum { kEpiF32 = 0, kEpiBf16 = 1, kEpiSwiglu = 2, kEpiSums = 3 };

struct I8GemmArgs {
  const int8_t* A;         // codes of the rows [.][K]
  const float* sa;         // their scales
  const int32_t* row_src;  // grouped: row of A of each sorted position (null: the position itself)
  const int4* tiles;       // grouped: {expert (-1 shared, -2 none), first position, rows, 0}; null: dense
  int64_t rows;            // dense: rows of A
  uint32_t a_rows;         // gathered: rows of A (a_rows * K at most 2^32 - 2^20)
  int64_t P;               // grouped: routed positions; position P + t is token t's for the shared expert
  int K, N;                // N output columns (SwiGLU: gate columns, as many up columns)
  I8Mat W, W2;             // weights (stacked by expert), SwiGLU: gate and up
  I8Mat S, S2;             // the shared expert's
  int n_slices;            // column slices of a tile
  int64_t tiles_n;         // row tiles
  void* out;               // [position][N]
};

constexpr int kStepBytes = 128;  // columns of a K step, one cache line of every operand row
// Tile rows of a band: the 32 workgroups that an XCD runs at a time then cover 4 x 8 tiles.
constexpr int kBand = 4;

__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }

template <typename F, int... St>
__device__ __forceinline__ void each_stage(F f, std::integer_sequence<int, St...>) {
  (f(std::integral_constant<int, St>{}), ...);
}

// Measured (MI355X; a large copy moves 5.1 TB/s, the library's int8 product of 8192^3 runs at
// 2.1 POP/s): 8192 x 8192 x 4096 in 233-266 us as the clock goes, 2.1-2.4 POP/s; its matrix
// instructions are busy 62% of that (177 us of them alone on this data), what is left is the
// loads' and the turn's share that they do not cover.
// Grouped, 16,384 rows over 256 experts of 2048 x 512 and 2,048 of the shared one: gate/up
// 136 us for 541 MB of weights (4.0 TB/s), down 92 us for 270 MB of weights and 151 MB of sums
// (4.6 TB/s): bound by these bytes, and by the last of 4.25 rounds of workgroups.
// Operand tiles of 64 x 64 per wave were taken for them over 128 x 64 (139 and 86 us against
// 131 and 80, half the waves) and over two smaller workgroups a compute unit (285 us a layer
// against 263), both with sums of two bytes.
//
// Workgroup = WM x WN waves, each FM x FN blocks of 32 x 32 (v_mfma_i32_32x32x32_i8).  Each
// 128-column K step of both operands goes through LDS by 16-byte DMA loads (8 lanes read a
// row's whole line) in kStages stages; inside a row the eight 16-byte pieces are
// XOR-rotated by row bits 1-3 so that the operand reads (a row per lane) spread over all
// banks.  K is a multiple of 64: where it is not one of 128 the last step's upper half is
// not multiplied (its bytes are the next row's, or zeros).
template <int WM, int WN, int FM, int FN, int kStages, int EPI>
__device__ __forceinline__ void i8_tile_body(const I8GemmArgs& p) {
  constexpr int TM = WM * FM * 32, TN = WN * FN * 32, kWaves = WM * WN;
  constexpr int kOps = (TM + TN) / 8 / kWaves;  // DMA loads per wave and step, 8 rows each
  static_assert((TM + TN) / 8 % kWaves == 0 && (kStages == 2 || kStages == 3), "whole blocks of 8 rows per wave");
  constexpr int kStageBytes = (TM + TN) * kStepBytes;
  // one array per stage, so that the compiler can tell a stage's reads from the loads
  // still filling another
  __shared__ __align__(16) uint8_t s_st0[kStageBytes], s_st1[kStageBytes], s_st2[kStages > 2 ? kStageBytes : 16];
  constexpr bool kSwiglu = EPI == kEpiSwiglu;
  constexpr int kCols = kSwiglu ? TN / 2 : TN;  // output columns of a tile
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;

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
    rows = min(TM, (int)(p.rows - first));
  }
  const I8Mat w = expert < 0 ? p.S : p.W, w2 = expert < 0 ? p.S2 : p.W2;
  const int64_t e_row = (int64_t)max(expert, 0) * p.N;  // first row of this expert's matrix

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
    int blk, row;  // block of 8 rows in the stage, row of the operand
    bool inside = true;
    if (j < kOpsA) {
      blk = wave * kOpsA + j;
      const int r = blk * 8 + (lane >> 3);
      row = r;
      if (p.row_src) {  // gathered rows: offsets from the whole matrix
        const int64_t pos = first + min(r, rows - 1);
        row = pos < p.P ? p.row_src[pos] : (int)(pos - p.P);
      }
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
    off[j] = inside ? (int)((uint32_t)row * (uint32_t)p.K + (uint32_t)(piece ^ row_swz(r)) * 16) : (int)0xFFFFFFF0u;
    dst[j] = blk * 8 * kStepBytes;
  }
  auto rsrc = [&](const int8_t* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base), 0, (int)bytes, kBufferRsrcWord3);
  };
  const int64_t w_off = (e_row + n0) * p.K;
  const uint32_t w_bytes = (uint32_t)min(kCols, p.N - n0) * (uint32_t)p.K;  // a tile's rows: at most 256 * 65536
  const __amdgpu_buffer_rsrc_t ra =
      rsrc(p.row_src ? p.A : p.A + first * p.K, (p.row_src ? p.a_rows : (uint32_t)rows) * (uint32_t)p.K);
  const __amdgpu_buffer_rsrc_t rw = rsrc(w.codes + w_off, w_bytes), ru = rsrc(w2.codes + w_off, w_bytes);
  auto stage = [&](int st) -> uint8_t* { return st == 0 ? s_st0 : st == 1 ? s_st1 : s_st2; };
  const int steps = (p.K + kStepBytes - 1) / kStepBytes;
  // steps past the last load it again and are not computed
  auto issue_op = [&](int i, int st, int j) __attribute__((always_inline)) {
    const int k0 = min(i, steps - 1) * kStepBytes;
    const __amdgpu_buffer_rsrc_t r = j < kOpsA ? ra : j < kOpsA + kOpsG ? rw : ru;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, stage(st) + dst[j], 16, off[j], k0, 0, 0);
  };

  // Operand reads run one MFMA step (32 columns) ahead of the products.  At the end of a K
  // step, with the last 32 columns' operands in registers, the workgroup meets: every wave
  // has read the stage, so its next loads go out, the next stage's first operands are read,
  // and the last products cover both.
  const int m = lane & 31, h = lane >> 5;
  i32x16_t acc[FM][FN] = {};
  auto run = [&](auto nf_c) __attribute__((always_inline)) {
    constexpr int NF = decltype(nf_c)::value;
    i32x4_t a[2][NF > 0 ? NF : 1], b[2][FN];
    auto read = [&](const uint8_t* base, int kk, int set) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);  // these reads go out before the products that follow in the source
      if constexpr (NF > 0) {
        const int c = 2 * kk + h;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const int r = (wm * FM + f) * 32 + m;
          a[set][f] = *reinterpret_cast<const i32x4_t*>(base + r * kStepBytes + ((c ^ row_swz(r)) << 4));
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          const int r = TM + (wn * FN + f) * 32 + m;
          b[set][f] = *reinterpret_cast<const i32x4_t*>(base + r * kStepBytes + ((c ^ row_swz(r)) << 4));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // One MFMA step, with the loads [j0, j1) of a K step into stage st between its products.
    auto mul = [&](int set, int i, auto st_c, auto j0_c, auto j1_c) __attribute__((always_inline)) {
      constexpr int st = decltype(st_c)::value, j0 = decltype(j0_c)::value, j1 = decltype(j1_c)::value;
      constexpr int kPer = (j1 - j0 + NF - 1) / (NF > 0 ? NF : 1);  // loads after each row of products
#pragma unroll
      for (int fm = 0; fm < NF; ++fm) {
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
          acc[fm][fn] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[set][fn], a[set][fm], acc[fm][fn], 0, 0, 0);
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
    using None = std::integral_constant<int, 0>;
    using Half = std::integral_constant<int, kOps / 2>;
    using All = std::integral_constant<int, kOps>;
    // kk = 0's operands are in set 0 on entry, and the next step's on return
    auto step = [&](int i, auto st_c) __attribute__((always_inline)) {
      constexpr int st = decltype(st_c)::value;
      using Free = std::integral_constant<int, (st + kStages - 1) % kStages>;  // the stage read before this one
      read(stage(st), 1, 1);
      mul(0, i + kStages - 1, Free{}, Half{}, All{});
      read(stage(st), 2, 0);
      mul(1, 0, st_c, None{}, None{});
      read(stage(st), 3, 1);
      mul(0, 0, st_c, None{}, None{});
      meet(std::integral_constant<int, kOps * (kStages - 2)>{});
      read(stage((st + 1) % kStages), 0, 0);
      mul(1, i + kStages, st_c, None{}, Half{});
    };
    meet(std::integral_constant<int, kOps * (kStages - 2) + kOps / 2>{});
    read(stage(0), 0, 0);
    const int full = p.K / kStepBytes;
    int i = 0;
    for (; i + kStages <= full; i += kStages)
      each_stage([&](auto st_c) { step(i + decltype(st_c)::value, st_c); }, std::make_integer_sequence<int, kStages>{});
    each_stage(
        [&](auto st_c) {
          if (i + decltype(st_c)::value < full) step(i + decltype(st_c)::value, st_c);
        },
        std::make_integer_sequence<int, kStages - 1>{});
    if (p.K % kStepBytes) {  // the last 64 columns
      read(stage(full % kStages), 1, 1);
      mul(0, 0, None{}, None{}, None{});
      mul(1, 0, None{}, None{}, None{});
    }
  };
#pragma unroll
  for (int st = 0; st < kStages; ++st)
#pragma unroll
    for (int j = 0; j < (st + 1 < kStages ? kOps : kOps / 2); ++j) issue_op(st, st, j);
  // grouped tiles are often part full: only the 32-row blocks that hold rows are multiplied
  if constexpr (EPI == kEpiF32 || EPI == kEpiBf16) {
    run(std::integral_constant<int, FM>{});
  } else {
    static_assert(FM == 2, "none, one or both of a wave's blocks");
    const int held = rows - wm * FM * 32;
    if (held > 32) run(std::integral_constant<int, 2>{});
    else if (held > 0) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
  }
  __builtin_amdgcn_s_waitcnt(0);  // the repeated loads of the last steps are still landing

  // The weight is the first operand of the products, so that a lane holds sums of one row of
  // A (lane % 32) and four consecutive output columns (8*(i/4) + 4*(lane/32) + i%4).  Stored
  // from there a column quad of 32 rows would touch 32 cache lines, at a power-of-two
  // distance for most N; so each wave turns 32 rows at a time in LDS and stores whole rows
  // of its columns, 16 bytes a lane.
  constexpr bool kHalf = EPI == kEpiBf16;
  typedef typename std::conditional<kHalf, uint16_t, float>::type out_t;
  constexpr int kOutF = kSwiglu ? FN / 2 : FN;
  constexpr int kRow = kOutF * 32 * sizeof(out_t), kPitch = kRow + 16;  // the pad spreads the rows over the banks
  constexpr int kVec = 16 / sizeof(out_t);
  static_assert(kWaves % 2 == 0 && kWaves / 2 * 32 * kPitch <= kStageBytes, "the waves' blocks fit two stages");
  uint8_t* turn = (wave < kWaves / 2 ? s_st0 : s_st1) + wave % (kWaves / 2) * 32 * kPitch;
  const bool whole = p.N % kVec == 0;  // 16 bytes of a row are inside or outside together, and aligned
  const int c0 = n0 + wn * kOutF * 32;
  __builtin_amdgcn_s_barrier();  // no wave reads the stages any more
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int r0 = (wm * FM + fm) * 32;
    if (r0 >= rows) break;
    float sa = 0.f;
    if constexpr (EPI != kEpiSums) {
      const int64_t pos = first + min(r0 + m, rows - 1);
      sa = p.sa[p.row_src ? (pos < p.P ? (int64_t)p.row_src[pos] : pos - p.P) : pos];
    }
#pragma unroll
    for (int fn = 0; fn < kOutF; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = fn * 32 + 8 * q + 4 * h;
        out_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float d = (float)acc[fm][fn][4 * q + j];
          const int64_t row = e_row + min(c0 + c + j, p.N - 1);
          if constexpr (kSwiglu) {
            const float g = i8_scaled(d, sa, w.scales[row]);
            const float u = i8_scaled((float)acc[fm][fn + FN / 2][4 * q + j], sa, w2.scales[row]);
            o[j] = i8_swiglu(g, u);
          } else if constexpr (EPI == kEpiSums) {
            o[j] = d;
          } else if constexpr (EPI == kEpiBf16) {
            o[j] = i8_bf16(d * sa * w.scales[row]);
          } else {
            o[j] = d * sa * w.scales[row];
          }
        }
        uint8_t* to = turn + m * kPitch + c * sizeof(out_t);
        if constexpr (kHalf)
          *reinterpret_cast<uint2*>(to) = make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
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

template <int WM, int WN, int FM, int FN, int kStages, int EPI>
__global__ __launch_bounds__(WM* WN* kWave) void i8_tile_kernel(I8GemmArgs p) {
  i8_tile_body<WM, WN, FM, FN, kStages, EPI>(p);
}

template <int WM, int WN, int FM, int FN, int kStages, int EPI>
hipError_t launch_tiles(I8GemmArgs p, int64_t tiles, hipStream_t stream) {
  constexpr int kCols = WN * FN * 32 / (EPI == kEpiSwiglu ? 2 : 1);
  p.n_slices = (p.N + kCols - 1) / kCols;
  p.tiles_n = tiles;
  const int64_t blocks = p.tiles ? (tiles + kXcds - 1) / kXcds * kXcds * p.n_slices
                                 : (tiles * p.n_slices + kXcds - 1) / kXcds * kXcds;
  if (blocks <= 0) return hipSuccess;
  if (blocks * (WM * WN * kWave) > kMaxThreads) return hipErrorInvalidValue;  // bounded by the callers
  hipLaunchKernelGGL((i8_tile_kernel<WM, WN, FM, FN, kStages, EPI>), dim3((unsigned)blocks), dim3(WM * WN * kWave), 0,
                     stream, p);
  return hipGetLastError();
}

// Bound by the sums' bytes, written just before: 151 MB for 2,048 tokens of 9 slots and 2,048
// columns in 34 us (4.7 TB/s with the rows written), beside the channels' scales from the L2.
// The sums stay in fp32: fp16 ones made the layer 261 us instead of 284, and a bf16 output less
// exact than its 8 bits where slots cancel.
// y[t] = sum_i (sums of slot i * its row's scale * the channel's scale) w_i + shared, in slot
// order, the shared expert last; slots whose id names no expert add nothing.
__global__ __launch_bounds__(256) void i8_combine_kernel(const float* __restrict__ part, const float* __restrict__ sh,
                                                         const int32_t* __restrict__ inv,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int64_t T, int k, int E,
                                                         int H, int64_t P, const float* __restrict__ sw,
                                                         const float* __restrict__ sw_shared, void* __restrict__ Y,
                                                         int out_bf16) {
  const int per = H / 8;
  const int64_t total = T * per;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per;
    const int n = (int)(i - t * per) * 8;
    float y[8] = {};
    auto add = [&](int64_t pos, float scale, float f, const float* s) {
      float c[8];
      const float4* q = reinterpret_cast<const float4*>(part + pos * H + n);
      const float v[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = s[n + j];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = i8_add_slot(y[j], i8_scaled(v[j], scale, c[j]), f);
    };
    for (int s0 = 0; s0 < k; s0 += 4) {  // four slots' loads in flight
      int e[4];
      int64_t pos[4];
      float f[4], scale[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = t * k + min(s0 + j, k - 1);
        e[j] = ids[r];
        pos[j] = s0 + j < k && e[j] >= 0 && e[j] < E ? inv[r] : -1;
        f[j] = weights[r];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) scale[j] = sh[pos[j] < 0 ? 0 : pos[j]];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (pos[j] >= 0) add(pos[j], scale[j], f[j], sw + (int64_t)e[j] * H);
    }
    if (sw_shared) add(P + t, sh[P + t], 1.0f, sw_shared);
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

constexpr int kExpertRows = 128;  // rows of a grouped tile

struct ExpertsWs {
  int8_t* xq;            // [T][H] codes of the tokens
  float* sx;             // [T]
  int32_t *offsets, *sorted, *inv, *row_src;
  float* row_w;
  int4* tiles;
  void* perm;
  float* act;            // [R][I] silu(gate) * up of each sorted position
  int8_t* aq;            // [R][I] its codes
  float* sh;             // [R]
  float* part;           // [R][H] sums of the down product
  size_t total;
};

ExpertsWs carve(void* base, const I8Experts& L, int64_t T, int k) {
  ExpertsWs w{};
  char* c = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) { char* r = c ? c + off : nullptr; off += align256(bytes); return r; };
  const int64_t P = T * k, extra = L.sh_gate.codes ? T : 0, R = P + extra;
  w.xq = reinterpret_cast<int8_t*>(take((size_t)T * L.hidden));
  w.sx = reinterpret_cast<float*>(take((size_t)T * 4));
  w.offsets = reinterpret_cast<int32_t*>(take((size_t)(L.n_experts + 1) * 4));
  w.sorted = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  w.inv = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  w.row_src = reinterpret_cast<int32_t*>(take((size_t)P * 4));
  w.row_w = reinterpret_cast<float*>(take((size_t)P * 4));
  w.tiles = reinterpret_cast<int4*>(take((size_t)group_max_tiles(P, L.n_experts, extra, kExpertRows) * 16));
  w.perm = take(permute_workspace_bytes(P, L.n_experts));
  w.act = reinterpret_cast<float*>(take((size_t)R * L.inter * 4));
  w.aq = reinterpret_cast<int8_t*>(take((size_t)R * L.inter));
  w.sh = reinterpret_cast<float*>(take((size_t)R * 4));
  w.part = reinterpret_cast<float*>(take((size_t)R * L.hidden * 4));
  w.total = off;
  return w;
}

}  // namespace

hipError_t run_i8_quantize(const uint16_t* X, int64_t rows, int K, int8_t* codes, float* scales, hipStream_t stream) {
  return launch_quantize(X, rows, K, codes, scales, stream);
}

size_t i8_gemm_workspace_bytes(int64_t m, int K) { return align256((size_t)m * K) + align256((size_t)m * 4); }

hipError_t run_i8_gemm(const I8Mat& W, int64_t n, int K, const uint16_t* X, int64_t m, void* Y, int out_bf16, void* ws,
                       hipStream_t stream) {
  if (i8_few_rows(m, K)) return run_i8_few_rows(W, n, K, X, (int)m, Y, out_bf16, stream);
  int8_t* xq = static_cast<int8_t*>(ws);
  float* sx = reinterpret_cast<float*>(static_cast<char*>(ws) + align256((size_t)m * K));
  hipError_t e = launch_quantize(X, m, K, xq, sx, stream);
  if (e != hipSuccess) return e;
  I8GemmArgs p{};
  p.A = xq;
  p.sa = sx;
  p.rows = m;
  p.K = K;
  p.N = (int)n;
  p.W = p.W2 = p.S = p.S2 = W;
  p.out = Y;
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

size_t experts_i8_workspace_bytes(const I8Experts& L, int64_t T, int k) {
  // a workspace made for T tokens also takes fewer, the few-slots form among them
  return std::max(carve(nullptr, L, T, k).total, align256(i8_few_slots_bytes(L, T, k)));
}

hipError_t run_moe_experts_i8(const I8Experts& L, const uint16_t* X, int64_t T, const int32_t* ids,
                              const float* weights, int k, void* Y, int out_bf16, void* ws, hipStream_t stream) {
  if (i8_few_slots(L, T, k))
    return run_i8_few_slots(L, X, (int)T, ids, weights, k, Y, out_bf16, static_cast<float*>(ws), stream);
  const int H = L.hidden, I = L.inter, E = L.n_experts;
  const ExpertsWs w = carve(ws, L, T, k);
  const int64_t P = T * k, extra = L.sh_gate.codes ? T : 0, R = P + extra;
  const int max_tiles = group_max_tiles(P, E, extra, kExpertRows);
  GroupTiles gt{};
  gt.tile_rows = kExpertRows;
  gt.max_tiles = max_tiles;
  gt.extra_rows = extra;
  gt.topk = k;
  gt.table = w.tiles;
  gt.row_src = w.row_src;
  gt.row_w = w.row_w;
  // the tokens' codes are made in the sort's first launch, beside its few workgroups
  const I8RowsJob job{X, T, H, w.xq, w.sx};
  hipError_t e = run_permute(ids, P, E, w.offsets, w.sorted, w.inv, w.perm, &gt, stream, nullptr, &job);
  if (e != hipSuccess) return e;

  I8GemmArgs p{};
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
  p.out = w.act;
  e = launch_tiles<2, 4, 2, 2, 3, kEpiSwiglu>(p, max_tiles, stream);
  if (e != hipSuccess) return e;
  e = launch_quantize(w.act, R, I, w.aq, w.sh, stream);
  if (e != hipSuccess) return e;

  I8GemmArgs d = p;
  d.A = w.aq;
  d.sa = w.sh;
  d.row_src = nullptr;
  d.K = I;
  d.N = H;
  d.W = d.W2 = L.down;
  d.S = d.S2 = L.sh_down;
  d.out = w.part;
  e = launch_tiles<2, 4, 2, 2, 3, kEpiSums>(d, max_tiles, stream);
  if (e != hipSuccess) return e;

  const unsigned blocks = (unsigned)std::min<int64_t>((T * (H / 8) + 255) / 256, 65536);
  hipLaunchKernelGGL(i8_combine_kernel, dim3(blocks), dim3(256), 0, stream, w.part, w.sh, w.inv, ids, weights, T, k, E, H,
                     P, L.down.scales, extra ? L.sh_down.scales : nullptr, Y, out_bf16);
  return hipGetLastError();
}

}  // namespace q4moe
