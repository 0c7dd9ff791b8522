// The next token of each row of logits, drawn by a given random number after temperature,
// top-k, top-p and min-p (sample_logits).
//
// Tokens are ordered by logit, the lower index first among equals; each filter keeps a first
// part of that order, so together they keep the shortest of them, and what is kept is told
// by one 50-bit word (the logit's ordered bits, then the index inverted): a token stays when
// its word is at least that of the last one kept.  The draw goes over the kept tokens in the
// vocabulary's order.
//
// Weights are integers, w = exp((l - max) / t) rounded to multiples of 2^-45 (from fp64), so
// sums are exact: no order of additions, split of a row or atomic add changes a result, and a
// row gets the same token in any batch.  A row of 2^18 tokens sums to at most 2^63.
//
// Up to three launches.  peak_kernel reads the logits once for the largest of every 64
// consecutive ones (a part) and of every chunk.  Where top-k rules, the k-th largest of the
// parts' maxima is a bound that at least k tokens reach, so one workgroup of front_kernel
// reads only the parts that reach it, lists their tokens in LDS, and finds the last
// token kept and the draw in the list.  A top-p without such a top-k needs the whole row's
// weights: other workgroups of front_kernel add them by bins of (max - l) / t (bins as fine as 2^-8
// of it) and find the bin in which the filter ends; row_kernel, on all chunks, adds up what
// lies above that bin for every 1,024 tokens (a step), lists the bin, and the last workgroup of
// the row to arrive finds the token.  Without either filter row_kernel adds up the steps.
// Steps whose parts' maxima reach nothing that is kept are not read.  Where a list would
// overflow (many equal logits) a workgroup selects from the row itself, digit by digit.
//
// Measured on 151,936 fp32 logits, whole calls in a graph: one row 14 us without a filter, 18 with
// top-k 50, 36 with a top-p of 0.9 alone; 256 rows 75, 42 and 167, of mixed parameters 102.  The first
// reading is bound by memory; a list's selection by latency (one workgroup a row); the bins by
// their atomic adds in LDS, the steps' sums by the fp64 of the weights (not told apart by counters).
// Rows whose list overflows are far slower (draw_alone).
#include <algorithm>
#include <type_traits>

#include "steps.h"
#include "wave64.h"

namespace q4moe {

namespace {

constexpr int kPart = 64;         // tokens of a part
constexpr int kStep = 1024;       // tokens of a step, one wave's at a time
constexpr int kMaxChunks = 128;   // of a row
constexpr int kMaxSteps = kMaxSampleVocab / kStep;
constexpr int kList = 2048;       // tokens of a row's list
constexpr int kTopMost = 1024;    // the largest top-k that goes by parts
constexpr int kBins = 4096;
constexpr int kDigits = 2048;     // of a selection's level
constexpr int kWordBits = 50, kIndexBits = 18;
constexpr uint64_t kIndexMask = (1ull << kIndexBits) - 1;
constexpr int kOneBits = 45;      // the largest logit's weight is 2^45
constexpr double kNone = kOneBits + 1;  // of 2^-46 of that and less nothing is left

static_assert(kMaxSampleVocab == 1 << kIndexBits, "an index fits its bits");

// A row's state between the launches.
struct RowState {
  unsigned band_arrived, row_arrived, listed, over;  // over: top-k's list overflowed
  float above, reach;           // logits above are kept by top-k and top-p, those from reach on are listed
  int banded;                   // 0: neither ends in the row, all are kept
  unsigned c_base;              // top-k: tokens above
  int k;                        // top-k among the tokens that have a weight, 0: none
  uint64_t w_base, total;       // weight of those above, and the row's
};

struct SampleArgs {
  const void* logits;
  int64_t B;
  int V;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t* ids;
  float* probs;
  int G, chunk, M;              // chunks of a row, tokens of a chunk, parts of a row
  uint64_t* peaks;              // [B][G] the chunk's largest word
  float* parts;                 // [B][M]
  uint32_t* counts;             // [B][kBins]
  uint64_t* weights;            // [B][kBins]
  uint64_t* sums;               // [B][kMaxSteps]
  uint64_t* list;               // [B][kList]
  RowState* state;              // [B]
};

enum Kind {
  kGreedy,
  kAll,   // a list of all tokens
  kTop,   // a list of the tokens that top-k, or min-p alone, may keep
  kBand,  // the band in which top-p or a large top-k ends
  kSum    // no filter
};

struct RowRule {
  Kind kind;
  double scale, limit;          // scale: log2(e) / t; limit: weights of 2^-limit and less drop
  float p, u;                   // top-p's share and the draw's number, in [0, 1]
  int k;                        // 0 without top-k
  bool p_on;
};

__device__ __forceinline__ RowRule row_rule(const SampleArgs& a, int64_t b) {
  RowRule r;
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.0f, m = a.min_p ? a.min_p[b] : 0.0f;
  const float u = a.u[b];
  r.u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;
  r.scale = 1.4426950408889634 / (double)t;
  r.k = k > 0 && k < a.V ? k : 0;
  r.p_on = p < 1.0f;
  r.p = p > 0.0f ? p : 0.0f;
  r.limit = kNone;
  if (m > 0.0f) {  // 2^-y >= m; the next number above, as what is kept lies below the limit
    const double most = fmax(-log2((double)m), 0.0);
    r.limit = fmin(kNone, __longlong_as_double(__double_as_longlong(most) + 1));
  }
  r.kind = !(t > 0.0f)                            ? kGreedy
           : a.V <= kList                         ? kAll
           : r.k ? (r.k <= min(a.M / 2, kTopMost) ? kTop : kBand)
           : r.p_on                               ? kBand
           : r.limit < kNone                      ? kTop
                                                  : kSum;
  return r;
}

// A logit as the rules take it: a NaN is closed as -infinity is, and both zeros are one.
__device__ __forceinline__ float clean(float l) { return l == l ? l + 0.0f : -__builtin_inff(); }

template <typename In>
__device__ __forceinline__ float as_logit(In raw) {
  if constexpr (sizeof(In) == 2) return clean(bf16_bits_to_f32(raw));
  else return clean(raw);
}

// 16 bytes of consecutive logits from i on; closed from `end` on.
template <typename In>
struct Logits {
  static constexpr int kPer = 16 / sizeof(In);
  In raw[kPer];
  __device__ __forceinline__ void load(const In* row, int i, int end) {
    if (i + kPer <= end) {
      __builtin_memcpy(raw, row + i, 16);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if constexpr (sizeof(In) == 2) raw[j] = i + j < end ? row[i + j] : (In)0xFF80;
        else raw[j] = i + j < end ? row[i + j] : -__builtin_inff();
      }
    }
  }
  __device__ __forceinline__ float at(int j) const { return as_logit(raw[j]); }
  // The same where a NaN and a zero's sign make no difference.
  __device__ __forceinline__ float as_is(int j) const {
    if constexpr (sizeof(In) == 2) return bf16_bits_to_f32(raw[j]);
    else return raw[j];
  }
};

// The place in the order: 50 bits, larger first.
__device__ __forceinline__ uint64_t word_of(float l, int i) {
  return (uint64_t)float_key(l) << kIndexBits | (kIndexMask - (uint64_t)i);
}
__device__ __forceinline__ int index_of(uint64_t word) { return (int)(kIndexMask - (word & kIndexMask)); }
__device__ __forceinline__ float logit_of(uint64_t word) { return key_float((uint32_t)(word >> kIndexBits)); }

// 2^(45 - j/256), the fractions of the weights' exponential.
constexpr int kPowers = 256;
struct Powers {
  double of[kPowers];
  __device__ __forceinline__ void fill() {
    if (threadIdx.x < kPowers) of[threadIdx.x] = exp2(kOneBits - (double)threadIdx.x / kPowers);
  }
};

// A row's weights.  kFinite (the row's largest logit is) leaves out what an infinite one needs.
struct Weights {
  const Powers* pow;
  double top, scale;
  float top_f, scale_f;
  __device__ __forceinline__ Weights(const Powers* powers, float top_, double scale_)
      : pow(powers), top((double)top_), scale(scale_), top_f(top_), scale_f(fminf((float)scale_, 3.402823466e38f)) {}  // (0 times it stays 0)
  __device__ __forceinline__ bool finite() const { return top_f < __builtin_inff(); }

  // (max - l) / t in powers of two; a NaN for closed logits under an infinite t or maximum.
  template <bool kFinite = false>
  __device__ __forceinline__ double distance(float l) const {
    const double y = (top - (double)l) * scale;
    return !kFinite && l == top_f ? 0.0 : y;
  }

  // Closed logits and those beyond 2^-46 of the largest have no weight, and change no
  // filter's end.
  __device__ __forceinline__ bool weighs(float l) const { return distance(l) < kNone; }

  // 0 from `limit` on, and for a NaN.  2^(45-y) for y = n / 256 + r: the table's value for n % 256
  // with n / 256 off its exponent, times exp(-r ln 2) by its series to the fourth power (|r| <= 2^-9:
  // 2^-54 of it is left out), rounded to an integer by the addition of 2^52: the sum's low bits.  No branches,
  // so that several run at once; what is computed beyond the limit is not used.
  template <bool kFinite = false>
  __device__ __forceinline__ uint64_t operator()(float l, double limit) const {
    const double y = distance<kFinite>(l);
    constexpr double kMagic = 6755399441055744.0 / kPowers;  // 1.5 * 2^52 steps of 1 / 256
    const double z = y + kMagic;
    const uint32_t n = (uint32_t)__double_as_longlong(z);
    const double r = y - (z - kMagic);
    constexpr double k1 = -0.69314718055994530942, k2 = k1 * k1 / 2, k3 = k2 * k1 / 3, k4 = k3 * k1 / 4;
    const double s = fma(fma(fma(fma(k4, r, k3), r, k2), r, k1), r, 1.0);
    const uint64_t t = (uint64_t)__double_as_longlong(pow->of[n % kPowers]);
    const uint64_t w = (uint64_t)__double_as_longlong(
        fma(__longlong_as_double((long long)pair64((uint32_t)t, (uint32_t)(t >> 32) - (n / kPowers << 20))), s, 4503599627370496.0));
    return y < limit ? pair64((uint32_t)w, (uint32_t)(w >> 32) & 0xFFFFFu) : 0;
  }

  // Bins of the distance, as fine as its exponent and 8 bits from 2^-10 to 2^6; they follow the
  // order of the logits.
  template <bool kFinite = false>
  __device__ __forceinline__ int bin(float l) const {
    const float v = (top_f - l) * scale_f, d = !kFinite && l == top_f ? 0.0f : v;
    constexpr int kFirst = (127 - 10) << 8;
    return min(max((int)(__float_as_uint(d) >> 15) - kFirst, 0), kBins - 1);
  }
};

__device__ __forceinline__ uint64_t ld64(const uint64_t* p) {
  return __hip_atomic_load(const_cast<uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st64(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void add64(uint64_t* lds, uint64_t v) {
  atomicAdd(reinterpret_cast<unsigned long long*>(lds), (unsigned long long)v);
}

// Whether this is the last of n workgroups to come here; what the others stored or added
// (device-coherently) before is then there to be read (device-coherently).
__device__ __forceinline__ bool last_to_arrive(unsigned* count, unsigned n) {
  __shared__ unsigned s_place;
  wait_vmem();
  __syncthreads();
  if (threadIdx.x == 0) s_place = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return s_place == n - 1;
}

// ---- the largest of every part and chunk
// Bound by the logits' bytes: 256 rows of 151,936 in fp32 in 26 us, 5.9 TB/s (156 MB, partly
// held by the last cache).  Also clears what the row's other launches count in.
constexpr int kPeakThreads = 256;
template <typename In>
__global__ __launch_bounds__(kPeakThreads) void peak_kernel(SampleArgs a) {
  constexpr int kPer = Logits<In>::kPer, kLanes = kPart / kPer;  // lanes to a part
  constexpr int kUnroll = 4, kThreads = kPeakThreads;
  __shared__ uint64_t s_best[kThreads / kWave];
  const int64_t b = blockIdx.x / a.G;
  const int g = blockIdx.x % a.G;
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  float* parts = a.parts + b * a.M;
  const int first = g * a.chunk, end = min(first + a.chunk, a.V);
  float best = -__builtin_inff();
  int at = first;
  for (int i0 = first + (int)threadIdx.x * kPer; i0 - (int)threadIdx.x * kPer < end; i0 += kUnroll * kThreads * kPer) {
    Logits<In> v[kUnroll];
#pragma unroll
    for (int o = 0; o < kUnroll; ++o) v[o].load(row, i0 + o * kThreads * kPer, end);
#pragma unroll
    for (int o = 0; o < kUnroll; ++o) {
      const int i = i0 + o * kThreads * kPer;
      float most = v[o].at(0);
#pragma unroll
      for (int j = 1; j < kPer; ++j) most = fmaxf(most, v[o].at(j));
      if (most > best) {  // the first of equals stays
        best = most;
        at = i;
#pragma unroll
        for (int j = kPer - 1; j >= 0; --j)
          if (v[o].at(j) == most) at = i + j;
      }
      float p = most;
      p = fmaxf(p, dpp_f32<kDppQuadXor1>(p));
      p = fmaxf(p, dpp_f32<kDppQuadXor2>(p));
      p = fmaxf(p, dpp_f32<kDppRowHalfMirror>(p));
      if constexpr (kLanes == 16) p = fmaxf(p, dpp_f32<kDppRowMirror>(p));
      if (threadIdx.x % kLanes == 0 && i < end) parts[i / kPart] = p;
    }
  }
  uint64_t w = wave_max_u64(word_of(best, at));
  if (lane_id() == 0) s_best[threadIdx.x / kWave] = w;
  lds_sync();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int o = 1; o < kThreads / kWave; ++o) w = max(w, s_best[o]);
    a.peaks[b * a.G + g] = w;
    if (g == 0) {
      a.state[b] = RowState{};
    }
  }
  if (row_rule(a, b).kind == kBand) {
    for (int i = g * kThreads + threadIdx.x; i < kBins; i += a.G * kThreads) {
      a.counts[b * kBins + i] = 0;
      a.weights[b * kBins + i] = 0;
    }
  }
}

// The row's largest word; every wave for itself.
__device__ __forceinline__ uint64_t row_peak(const SampleArgs& a, int64_t b) {
  static_assert(kMaxChunks == 2 * kWave, "two a lane");
  const int i = lane_id();
  const uint64_t v = i < a.G ? a.peaks[b * a.G + i] : 0, w = i + kWave < a.G ? a.peaks[b * a.G + i + kWave] : 0;
  return wave_max_u64(max(v, w));
}

// Sums before a thread over the workgroup's kThreads, and their total.
struct Pair {
  uint32_t c;
  uint64_t w;
};
template <int kThreads>
__device__ __forceinline__ Pair block_before(Pair mine, Pair* total) {
  constexpr int kWaves = kThreads / kWave;
  __shared__ uint32_t s_c[kWaves];
  __shared__ uint64_t s_w[kWaves];
  const int wave = threadIdx.x / kWave;
  const Pair in{wave_prefix(mine.c), wave_prefix(mine.w)};
  lds_sync();  // an earlier call's totals are read
  if (lane_id() == kWave - 1) {
    s_c[wave] = in.c;
    s_w[wave] = in.w;
  }
  lds_sync();
  Pair before{in.c - mine.c, in.w - mine.w}, all{0, 0};
#pragma unroll
  for (int o = 0; o < kWaves; ++o) {
    if (o < wave) {
      before.c += s_c[o];
      before.w += s_w[o];
    }
    all.c += s_c[o];
    all.w += s_w[o];
  }
  *total = all;
  return before;
}
template <int kThreads>
__device__ __forceinline__ uint64_t block_sum(uint64_t mine) {
  __shared__ uint64_t s_w[kThreads / kWave];
  mine = wave_sum_u64(mine);
  lds_sync();  // an earlier call's are read
  if (lane_id() == 0) s_w[threadIdx.x / kWave] = mine;
  lds_sync();
  uint64_t all = 0;
#pragma unroll
  for (int o = 0; o < kThreads / kWave; ++o) all += s_w[o];
  return all;
}

// The whole part of x n for x in [0, 1), and whether something is left: exactly, as a total has up to 63
// bits, ten more than fp64 holds.
struct Share {
  uint64_t whole;
  bool rest;
};
__device__ __forceinline__ Share share(float x, uint64_t n) {
  const uint32_t bits = __float_as_uint(x);
  const int down = 150 - (int)(bits >> 23);  // x is a whole number of 24 bits by 2^-down, 24 and more
  const uint64_t m = (bits & 0x7FFFFFu) | 0x800000u, lo = m * n, hi = __umul64hi(m, n);
  if (down >= 88 || x == 0.0f) return Share{0, x > 0.0f && n > 0};  // (subnormal numbers among them)
  if (down >= 64) return Share{hi >> (down - 64), (lo | (hi & ((1ull << (down - 64)) - 1))) != 0};
  return Share{hi << (64 - down) | lo >> down, (lo & ((1ull << down) - 1)) != 0};
}

// The least whole number that is at least p z, and 1 at least: a sum reaches p z when it
// reaches this.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t z) {
  const Share s = share(p, z);
  return max(s.whole + s.rest, (uint64_t)1);
}

// The draw's place among `total` of weight: the chosen token's running sum is the first beyond it.
__device__ __forceinline__ uint64_t mark_of(const RowRule& r, uint64_t total) {
  return r.u < 1.0f ? share(r.u, total).whole : total - 1;
}

__device__ __forceinline__ void answer(const SampleArgs& a, int64_t b, int id, double prob) {
  a.ids[b] = id;
  if (a.probs) a.probs[b] = (float)prob;
}

// ---- selection among words
struct Levels {
  uint64_t w[kDigits];
  uint32_t c[kDigits];
  uint64_t found_w;
  uint32_t found_c;
  int at;
};

// The word at which the count or the weight of the words from the largest on reaches its mark:
// need_c words, or need_w of weight.  each(visit) calls visit(word, weight) for this thread's share
// of the words; `bits` of them are compared, by digits of at most 11.  Returns a word that
// all kept ones reach and no others (of those visited), its untold bits zero, and in `with` what is
// kept.
template <int kThreads, typename Each>
__device__ __forceinline__ uint64_t select_word(Levels& s, int bits, uint32_t need_c, uint64_t need_w, Each each,
                                                Pair* with) {
  uint64_t prefix = 0;
  Pair above{0, 0};
  const uint64_t mask = (1ull << bits) - 1;
  int left = bits;
  while (true) {
    const int take = min(left, left > 18 ? 11 : 9);
    const int rest = left - take;
    for (int i = threadIdx.x; i < kDigits; i += kThreads) {
      s.w[i] = 0;
      s.c[i] = 0;
    }
    if (threadIdx.x == 0) s.at = -1;
    lds_sync();
    each([&](uint64_t word, uint64_t w) {
      word &= mask;
      if (word >> left != prefix) return;
      const int d = (int)(word >> rest) & ((1 << take) - 1);
      add64(&s.w[d], w);
      atomicAdd(&s.c[d], 1u);
    });
    lds_sync();
    // digits from the largest down
    constexpr int kOwn = kDigits / kThreads;
    const int own = kDigits - 1 - (int)threadIdx.x * kOwn;
    Pair mine{0, 0}, total;
    for (int i = 0; i < kOwn; ++i) {
      mine.c += s.c[own - i];
      mine.w += s.w[own - i];
    }
    Pair at = block_before<kThreads>(mine, &total);
    at.c += above.c;
    at.w += above.w;
    for (int i = 0; i < kOwn; ++i) {
      const Pair in{s.c[own - i], s.w[own - i]};
      const Pair up{at.c + in.c, at.w + in.w};
      // the mark is reached here, or with the last of the words where it is beyond them all
      const bool reached = need_c ? at.c < need_c && up.c >= need_c : at.w < need_w && up.w >= need_w;
      const bool end = in.c && up.c == above.c + total.c && (need_c ? up.c < need_c : up.w < need_w);
      if (reached || end) {
        s.at = own - i;
        s.found_c = at.c;
        s.found_w = at.w;
      }
      at = up;
    }
    lds_sync();
    const int d = s.at;
    if (d < 0) {  // no word at all
      *with = above;
      lds_sync();
      return 0;
    }
    above = Pair{s.found_c, s.found_w};
    const Pair in{s.c[d], s.w[d]};
    *with = Pair{above.c + in.c, above.w + in.w};
    prefix = prefix << take | (uint64_t)d;
    left = rest;
    lds_sync();
    if (left == 0 || in.c == 1 || (need_c && with->c == need_c)) return prefix << left;
  }
}

template <int kThreads>
__device__ __forceinline__ uint64_t block_or(uint64_t mine) {
  __shared__ uint64_t s_w[kThreads / kWave];
  mine = wave_reduce_u64(mine, [](uint64_t a, uint64_t b) { return a | b; });
  lds_sync();  // an earlier call's are read
  if (lane_id() == 0) s_w[threadIdx.x / kWave] = mine;
  lds_sync();
#pragma unroll
  for (int o = 0; o < kThreads / kWave; ++o) mine |= s_w[o];
  return mine;
}
template <int kThreads>
__device__ __forceinline__ uint64_t block_min(uint64_t mine) {
  __shared__ uint64_t s_w[kThreads / kWave];
  mine = wave_max_u64(~mine);
  lds_sync();  // an earlier call's are read
  if (lane_id() == 0) s_w[threadIdx.x / kWave] = mine;
  lds_sync();
#pragma unroll
  for (int o = 0; o < kThreads / kWave; ++o) mine = max(mine, s_w[o]);
  return ~mine;
}

// Up to so many tokens are compared with each other (n^2 / 8 cycles), more are told apart by
// digits (some us each selection, whatever the number).  One row and 256 rows of 151,936, top-k
// 100 with a top-p: 16.8 and 41.9 us against 19.0 and 47.1 by digits; top-k 200: 20.9 and 46.1
// against 19.3 and 46.1, with a top-p 21.4 and 46.6 against 23.1 and 49.9; top-k 400 compared
// 34.2 and 60.2 against 24.0 and 50.8.
constexpr int kRanked = 256;

// What a list is decided with; the list has room for 8 words more than it holds.
union Scratch {
  Levels levels;
  struct {
    alignas(16) uint64_t w[kRanked + 8];
    uint64_t heavier[kRanked];
    uint32_t place[kRanked];
  } rank;
};

// The word of the last token that the filters keep, from a list of n words: all tokens
// from the one after the first base.c of the order (their weight base.w) on, down to
// the last that top-k may keep or, without top-k, to the end of the row (z = 0) or of the bin in
// which top-p ends (z: the row's weight).
template <int kThreads>
__device__ __forceinline__ uint64_t last_kept(Scratch& s, uint64_t* list, int n, int k, bool p_on, float p,
                                              const Weights& weight, Pair base, uint64_t z) {
  if (n <= kRanked) {
    // A token's place and the weight before it by comparison with all others: a token a thread, or
    // as many threads to a token as there are, each with a slice of the others, eight at a time.
    int across = kWave;
    while (across < n) across *= 2;
    const int slices = kThreads / across, slice = threadIdx.x / across, i = threadIdx.x % across;
    const int len = ((n + slices - 1) / slices + 7) & ~7, from = slice * len, to = min(from + len, n);
    const uint64_t word = i < n ? list[i] : 0, w = i < n ? weight(logit_of(word), kNone) : 0;
    lds_sync();
    if (slice == 0) {
      s.rank.w[i] = w;
      s.rank.place[i] = base.c;
      s.rank.heavier[i] = base.w;
    }
    if (threadIdx.x < 8) {  // behind the last of the eights
      list[n + threadIdx.x] = 0;
      s.rank.w[across + threadIdx.x] = 0;
    }
    lds_sync();
    if (i - lane_id() < n && from < to) {
      uint32_t place = 0;
      uint64_t heavier = 0;
      for (int j = from; j < to; j += 8) {
        ulonglong2 q[4], v[4];
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          q[o] = *reinterpret_cast<const ulonglong2*>(&list[j + 2 * o]);
          v[o] = *reinterpret_cast<const ulonglong2*>(&s.rank.w[j + 2 * o]);
        }
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          place += q[o].x > word;
          place += q[o].y > word;
          heavier += q[o].x > word ? v[o].x : 0;
          heavier += q[o].y > word ? v[o].y : 0;
        }
      }
      if (i < n) {
        atomicAdd(&s.rank.place[i], place);
        add64(&s.rank.heavier[i], heavier);
      }
    }
    lds_sync();
    const uint32_t place = s.rank.place[i];
    const uint64_t heavier = s.rank.heavier[i];
    bool kept = i < n && slice == 0 && (!k || place < (uint32_t)k);
    if (p_on) {
      if (k || z == 0) z = base.w + block_sum<kThreads>(kept ? w : 0);
      kept = kept && heavier < share_of(p, z);
    }
    return block_min<kThreads>(kept ? word : ~0ull);
  }
  auto each = [&](auto visit) {
    for (int i = threadIdx.x; i < n; i += kThreads) visit(list[i], weight(logit_of(list[i]), kNone));
  };
  // from the first bit on in which the words differ
  uint64_t word = 0, differ = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) differ |= list[i] ^ list[0];
  const int bits = 64 - __clzll((long long)(block_or<kThreads>(differ) | 1));
  const uint64_t common = list[0] >> bits << bits;
  Pair with;
  if (k && (uint32_t)k < base.c + n) {
    word = common | select_word<kThreads>(s.levels, bits, k - base.c, 0, each, &with);
    z = base.w + with.w;
  } else if (k || z == 0) {  // all of them
    uint64_t mine = 0;
    each([&](uint64_t, uint64_t w) { mine += w; });
    z = base.w + block_sum<kThreads>(mine);
  }
  if (p_on) {
    const uint64_t need = share_of(p, z);
    word = max(word, common | select_word<kThreads>(s.levels, bits, 0, need > base.w ? need - base.w : 1, each, &with));
  }
  // that word tells the list's tokens apart: the last one's own
  uint64_t last = ~0ull;
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (list[i] >= word) last = min(last, list[i]);
  return block_min<kThreads>(last);
}

// ---- the second launch: rows that a list decides, and the bins of those that need them
constexpr int kFrontThreads = 512, kFrontWaves = kFrontThreads / kWave;

struct BandShared {
  uint64_t w[kBins];
  uint32_t c[kBins];
  Pair before;
  int bin;
  uint32_t edge[2];
};

struct PickShared {
  alignas(16) uint64_t list[kList + 8];
  union {
    Scratch scratch;
    uint32_t bins[kBins];
    uint16_t parts[kBins];
  };
  uint64_t word[kFrontWaves];
  alignas(16) uint32_t found[kFrontWaves];
  int at;
};
static_assert(kFrontWaves == 8, "found is read by fours");

// Appends a wave's words to the list; what is beyond its end is counted only.
template <int kN>
__device__ __forceinline__ void append(uint64_t* list, unsigned* n, const bool (&want)[kN], const uint64_t (&word)[kN]) {
  uint64_t ball[kN];
  uint32_t all = 0;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    ball[j] = __ballot(want[j]);
    all += __popcll(ball[j]);
  }
  if (all == 0) return;
  uint32_t base = 0;
  if (lane_id() == 0) base = atomicAdd(n, all);
  base = __builtin_amdgcn_readfirstlane(base);
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const uint32_t at = base + __popcll(ball[j] & ((1ull << lane_id()) - 1ull));
    if (want[j] && at < kList) list[at] = word[j];
    base += __popcll(ball[j]);
  }
}

// The draw from a list that holds every token kept, in the vocabulary's order.
__device__ __forceinline__ void draw_from_list(PickShared& s, int n, const SampleArgs& a, int64_t b, const RowRule& r,
                                               const Weights& weight) {
  constexpr int kThreads = kFrontThreads, kOwn = kList / kThreads;
  const uint64_t last =
      r.k || r.p_on ? last_kept<kThreads>(s.scratch, s.list, n, r.k, r.p_on, r.p, weight, Pair{0, 0}, 0) : 0;
  // the running sum, kOwn tokens a thread
  uint64_t word[kOwn], w[kOwn];
  Pair mine{0, 0}, total;
  const int own = n <= kThreads ? 1 : kOwn;
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const int i = threadIdx.x * own + o;
    word[o] = o < own && i < n ? s.list[i] : 0;
    w[o] = o < own && i < n && word[o] >= last ? weight(logit_of(word[o]), r.limit) : 0;
    mine.w += w[o];
  }
  uint64_t before = block_before<kThreads>(mine, &total).w;
  const uint64_t t = mark_of(r, total.w);
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    if (before <= t && before + w[o] > t) answer(a, b, index_of(word[o]), (double)w[o] / (double)total.w);
    before += w[o];
  }
}

template <typename In>
__device__ __forceinline__ void pick(PickShared& s, Powers& powers, const SampleArgs& a, int64_t b) {
  constexpr int kThreads = kFrontThreads;
  constexpr int kOwnParts = kMaxSampleVocab / kPart / kThreads, kOwnAll = kList / kThreads;
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const bool small = a.V <= kList;
  // What the row may need is on its way while its rule is read: consecutive tokens or parts a thread.
  // (Loads under a condition would wait for each other: indexes are kept inside instead.)
  float l[kOwnParts > kOwnAll ? kOwnParts : kOwnAll];
  if (small) {
    In raw[kOwnAll];
#pragma unroll
    for (int o = 0; o < kOwnAll; ++o) raw[o] = row[min((int)threadIdx.x * kOwnAll + o, a.V - 1)];
#pragma unroll
    for (int o = 0; o < kOwnAll; ++o)
      l[o] = (int)threadIdx.x * kOwnAll + o < a.V ? as_logit(raw[o]) : -__builtin_inff();
  } else {
#pragma unroll
    for (int o = 0; o < kOwnParts; ++o) l[o] = a.parts[b * a.M + min((int)threadIdx.x * kOwnParts + o, a.M - 1)];
#pragma unroll
    for (int o = 0; o < kOwnParts; ++o)
      if ((int)threadIdx.x * kOwnParts + o >= a.M) l[o] = -__builtin_inff();
  }
  uint64_t peak = small ? 0 : row_peak(a, b);
  const RowRule r = row_rule(a, b);
  if (r.kind == kBand || r.kind == kSum) return;
  powers.fill();
  if (small) {
#pragma unroll
    for (int o = 0; o < kOwnAll; ++o) {
      const int i = threadIdx.x * kOwnAll + o;
      if (i < a.V) peak = max(peak, word_of(l[o], i));
    }
    peak = wave_max_u64(peak);
    if (lane == 0) s.word[wave] = peak;
    lds_sync();
#pragma unroll
    for (int o = 0; o < kFrontWaves; ++o) peak = max(peak, s.word[o]);
  }
  const float top = logit_of(peak);
  if (r.kind == kGreedy || top == -__builtin_inff()) {
    const bool open = top != -__builtin_inff();
    if (threadIdx.x == 0) answer(a, b, open ? index_of(peak) : -1, open ? 1.0 : 0.0);
    return;
  }
  const Weights weight(&powers, top, r.scale);
  Pair mine{0, 0}, total;

  if (r.kind == kAll) {
#pragma unroll
    for (int o = 0; o < kOwnAll; ++o) mine.c += weight.weighs(l[o]);
    uint32_t at = block_before<kThreads>(mine, &total).c;
#pragma unroll
    for (int o = 0; o < kOwnAll; ++o)
      if (weight.weighs(l[o])) s.list[at++] = word_of(l[o], threadIdx.x * kOwnAll + o);
    lds_sync();
    draw_from_list(s, (int)total.c, a, b, r, weight);
    return;
  }

  // The parts whose largest token is kept where min-p rules; for top-k those that reach the bin
  // of the k-th largest of them.
  int bin[kOwnParts], bound = kBins - 1;
#pragma unroll
  for (int o = 0; o < kOwnParts; ++o)
    bin[o] = weight.distance(l[o]) < (r.k ? kNone : r.limit) ? weight.bin(l[o]) : kBins;
  if (r.k) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.bins[i] = 0;
    if (threadIdx.x == 0) s.at = kBins - 1;  // fewer parts than k hold a token of any weight
    lds_sync();
#pragma unroll
    for (int o = 0; o < kOwnParts; ++o)
      if (bin[o] < kBins) atomicAdd(&s.bins[bin[o]], 1u);
    lds_sync();
    constexpr int kOwn = kBins / kThreads;
    uint32_t in[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) mine.c += in[i] = s.bins[threadIdx.x * kOwn + i];
    uint32_t c = block_before<kThreads>(mine, &total).c;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (c < (uint32_t)r.k && c + in[i] >= (uint32_t)r.k) s.at = threadIdx.x * kOwn + i;
      c += in[i];
    }
    lds_sync();
    bound = s.at;
  }
  // These parts, in order, and the least of their maxima: at least k tokens reach that.  Without
  // k parts, and for min-p, every token that may be kept (and some that may not, which do not matter).
  mine.c = 0;
  uint32_t least = ~0u;
#pragma unroll
  for (int o = 0; o < kOwnParts; ++o) {
    mine.c += bin[o] <= bound;
    if (bin[o] <= bound) least = min(least, float_key(l[o]));
  }
  uint32_t at = block_before<kThreads>(mine, &total).c;
#pragma unroll
  for (int o = 0; o < kOwnParts; ++o)
    if (bin[o] <= bound) s.parts[at++] = (uint16_t)(threadIdx.x * kOwnParts + o);
  least = (uint32_t)block_min<kThreads>(least);  // (its barriers are behind the parts' writes)
  const int parts = (int)total.c;
  const float reach = fmaxf(parts < r.k || !r.k ? top - (float)((r.k ? kNone : r.limit) / r.scale) * 1.0001f - fabsf(top) * 1e-6f : key_float(least), -3.402823466e38f);
  // Their tokens that do, in order: 16 bytes a lane, so a load covers kPer parts, kLoads of them
  // at a time and the next ones on their way (the barriers wait for LDS alone).
  constexpr int kPer = Logits<In>::kPer, kLanes = kPart / kPer, kLoads = 4, kTurn = kFrontWaves * kLoads * kPer;
  uint32_t n = 0;
  Logits<In> next[kLoads];
  // A lane's first token, moved back where its 16 bytes would pass the row's end; tokens before `from` are
  // another lane's.
  auto tokens = [&](int o, int u, int* from) {
    *from = s.parts[min(o + u * kPer + lane / kLanes, parts - 1)] * kPart + lane % kLanes * kPer;
    return min(*from, a.V - kPer);
  };
  auto fetch = [&](int o) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      int from;
      __builtin_memcpy(next[u].raw, row + tokens(o, u, &from), 16);
    }
  };
  fetch(wave * kLoads * kPer);
  for (int o0 = 0; o0 < parts; o0 += kTurn) {
    const int o = o0 + wave * kLoads * kPer;
    Logits<In> v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) v[u] = next[u];
    if (o0 + kTurn < parts) fetch(o + kTurn);
    uint32_t want[kLoads], before[kLoads], all = 0;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      int from;
      const int i = tokens(o, u, &from);
      want[u] = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) want[u] |= (uint32_t)(v[u].at(j) >= reach && i + j >= from) << j;
      if (o + u * kPer + lane / kLanes >= parts) want[u] = 0;
      const uint32_t here = __popc(want[u]), upto = wave_prefix(here);
      before[u] = all + upto - here;
      all += __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    if (o0 > 0) lds_sync();  // the last turn's counts are read
    if (lane == 0) s.found[wave] = all;
    lds_sync();
    uint32_t to = n, found[kFrontWaves];
    *reinterpret_cast<uint4*>(found) = *reinterpret_cast<const uint4*>(s.found);
    *reinterpret_cast<uint4*>(found + 4) = *reinterpret_cast<const uint4*>(s.found + 4);
#pragma unroll
    for (int j = 0; j < kFrontWaves; ++j) {
      to += j < wave ? found[j] : 0;
      n += found[j];
    }
    n = __builtin_amdgcn_readfirstlane(n);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      int from;
      const int i = tokens(o, u, &from);
      uint32_t at = to + before[u];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (want[u] >> j & 1) {
          if (at < kList) s.list[at] = word_of(v[u].at(j), i + j);
          ++at;
        }
    }
    if (n > kList) break;
  }
  lds_sync();
  if (n <= kList) draw_from_list(s, (int)n, a, b, r, weight);
  else if (threadIdx.x == 0) a.state[b].over = 1;  // row_kernel's
}

template <typename In>
__device__ __forceinline__ void band(BandShared& s, Powers& powers, const SampleArgs& a, int64_t b, int g) {
  constexpr int kThreads = kFrontThreads, kPer = Logits<In>::kPer;
  const RowRule r = row_rule(a, b);
  if (r.kind != kBand) return;
  const float top = logit_of(row_peak(a, b));
  if (top == -__builtin_inff()) return;
  powers.fill();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.w[i] = 0;
    s.c[i] = 0;
  }
  lds_sync();
  const Weights weight(&powers, top, r.scale);
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  const int end = min((g + 1) * a.chunk, a.V);
  auto all = [&](auto finite) {
    constexpr bool kFinite = decltype(finite)::value;
    for (int i = g * a.chunk + (int)threadIdx.x * kPer; i < end; i += kThreads * kPer) {
      Logits<In> v;
      v.load(row, i, end);
      uint64_t w[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) w[j] = weight.template operator()<kFinite>(v.as_is(j), kNone);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (w[j] == 0) continue;
        const int bin = weight.template bin<kFinite>(v.as_is(j));
        add64(&s.w[bin], w[j]);
        if (r.k) atomicAdd(&s.c[bin], 1u);
      }
    }
  };
  if (weight.finite()) all(std::true_type{});
  else all(std::false_type{});
  lds_sync();
  uint32_t* counts = a.counts + b * kBins;
  uint64_t* weights = a.weights + b * kBins;
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    if (s.w[i] == 0) continue;
    __hip_atomic_fetch_add(&weights[i], s.w[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (r.k) __hip_atomic_fetch_add(&counts[i], s.c[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (!last_to_arrive(&a.state[b].band_arrived, a.G)) return;

  // the row's bins, and the ones in which the filters end
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.w[i] = ld64(&weights[i]);
    s.c[i] = r.k ? __hip_atomic_load(&counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
  }
  lds_sync();
  constexpr int kOwn = kBins / kThreads;
  const int own = threadIdx.x * kOwn;
  Pair mine{0, 0}, total;
  for (int i = 0; i < kOwn; ++i) {
    mine.c += s.c[own + i];
    mine.w += s.w[own + i];
  }
  const Pair before = block_before<kThreads>(mine, &total);
  // the first bin with which the count or the weight reaches its mark, and what lies before it
  auto find = [&](uint32_t need_c, uint64_t need_w, Pair* base) {
    Pair at = before;
    for (int i = 0; i < kOwn; ++i) {
      const Pair with{at.c + s.c[own + i], at.w + s.w[own + i]};
      const bool reached = need_c ? at.c < need_c && with.c >= need_c : at.w < need_w && with.w >= need_w;
      if (reached) {
        s.bin = own + i;
        s.before = at;
      }
      at = with;
    }
    lds_sync();
    const int bin = s.bin;
    *base = s.before;
    lds_sync();
    return bin;
  };
  const int k = r.k && (uint32_t)r.k <= total.c ? r.k : 0;
  int lo = kBins, hi = kBins;
  Pair base = total;
  uint64_t z = total.w;
  if (k) {
    lo = hi = find((uint32_t)k, 0, &base);
    z = base.w;  // what top-k keeps is at least that
  }
  if (r.p_on && z > 0) {
    lo = find(0, share_of(r.p, z), &base);
    if (!k) hi = lo;
  } else if (r.p_on) {  // the first bin has the end of both
    lo = 0;
    base = Pair{0, 0};
  }
  // the least logits of the bins before lo and up to hi: their keys bit by bit, as bins follow the logits
  if (threadIdx.x < 2) {
    const int most = threadIdx.x ? hi : lo - 1;
    uint32_t key = 0;  // the largest below which a logit's bin is beyond `most`
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t up = key | 1u << bit;
      const float l = key_float(up);
      if (up <= float_key(top) && (!(l > -__builtin_inff()) || weight.bin(l) > most)) key = up;
    }
    s.edge[threadIdx.x] = key;
  }
  lds_sync();
  if (threadIdx.x == 0) {  // read by the next launch
    RowState* st = &a.state[b];
    st->banded = lo < kBins;
    st->above = key_float(s.edge[0]);
    st->reach = key_float(s.edge[1] + 1);
    st->c_base = base.c;
    st->k = k;
    st->w_base = base.w;
    st->total = total.w;
  }
}

// Workgroups 0 .. rows - 1: a row each; the others: a chunk's bins.
template <typename In>
__global__ __launch_bounds__(kFrontThreads, 4) void front_kernel(SampleArgs a, unsigned rows) {
  __shared__ union Shared {
    BandShared band;
    PickShared pick;
    __device__ Shared() {}
  } s;
  __shared__ Powers powers;
  if (blockIdx.x < rows) pick<In>(s.pick, powers, a, blockIdx.x);
  else band<In>(s.band, powers, a, (blockIdx.x - rows) / a.G, (blockIdx.x - rows) % a.G);
}

// ---- the third launch: rows by the sums of their steps
constexpr int kRowThreads = 512, kRowWaves = kRowThreads / kWave;
static_assert(kMaxSteps <= kRowThreads, "a thread for each step's sum");

struct RowShared {
  alignas(16) uint64_t list[kList + 8];
  Scratch scratch;
  uint64_t sums[kMaxSteps];
  float queue[kRowWaves][2 * kWave];
  uint64_t found_w;
  unsigned n, base;
  int at;
};

// The draw from a row whose steps' sums of kept weights are in s.sums: a kept token is one whose
// word is at least `last`.
template <typename In>
__device__ __forceinline__ void draw_from_steps(RowShared& s, const SampleArgs& a, int64_t b, const RowRule& r,
                                                const Weights& weight, uint64_t last) {
  constexpr int kPer = Logits<In>::kPer, kLoads = kStep / kWave / kPer;
  const int steps = (a.V + kStep - 1) / kStep, lane = lane_id();
  const Pair mine{0, (int)threadIdx.x < steps ? s.sums[threadIdx.x] : 0};
  Pair total;
  const Pair at = block_before<kRowThreads>(mine, &total);
  uint64_t t = mark_of(r, total.w);
  if (at.w <= t && at.w + mine.w > t) {
    s.at = threadIdx.x;
    s.found_w = at.w;
  }
  lds_sync();
  if (threadIdx.x >= kWave) return;
  t -= s.found_w;
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  Logits<In> v[kLoads];
#pragma unroll
  for (int o = 0; o < kLoads; ++o) v[o].load(row, s.at * kStep + (o * kWave + lane) * kPer, a.V);
#pragma unroll
  for (int o = 0; o < kLoads; ++o) {
    const int i = s.at * kStep + (o * kWave + lane) * kPer;
    uint64_t w[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float l = v[o].at(j);
      sum += w[j] = word_of(l, i + j) >= last ? weight(l, r.limit) : 0;
    }
    uint64_t up = wave_prefix(sum), before = up - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (before <= t && before + w[j] > t) answer(a, b, i + j, (double)w[j] / (double)total.w);
      before += w[j];
    }
    up = __shfl(up, kWave - 1, kWave);
    if (t < up) break;  // uniform
    t -= up;
  }
}

// The draw by this workgroup alone: the last token kept by digits of the row's words, then the steps' sums.
// z: the row's weight, for a top-p without top-k.
// Up to five readings of the row for each filter and one more, every token's weight taken each time and
// most of them added to few counters: 151,936 logits in 0.6-1.1 ms, where a list takes 20-40 us.  Rows of many
// equal logits come here, bf16 ones away from zero among them (of mean 10 to 20 and a deviation of 1 to 2,
// under a top-p of 0.9 alone, more than 2,048 tokens share the logit in which p ends: one row 0.60-0.66 ms,
// 64 rows 1.1-1.3, 256 rows 2.2-2.3), rows under a top-p far inside a large top-k (5,000, p 0.9: 256 rows
// 1.8 ms), and rows of one value (one row 1.1 ms, 256 rows 4.6).
template <typename In>
__device__ __forceinline__ void draw_alone(RowShared& s, const SampleArgs& a, int64_t b, const RowRule& r, int k,
                                        const Weights& weight, uint64_t z) {
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  auto each = [&](auto visit) {
    for (int i = threadIdx.x; i < a.V; i += kRowThreads) {
      const float l = as_logit(row[i]);
      if (const uint64_t w = weight(l, kNone)) visit(word_of(l, i), w);
    }
  };
  uint64_t last = 0;
  Pair with;
  if (k) {
    last = select_word<kRowThreads>(s.scratch.levels, kWordBits, k, 0, each, &with);
    z = with.w;
  }
  if (r.p_on) last = max(last, select_word<kRowThreads>(s.scratch.levels, kWordBits, 0, share_of(r.p, z), each, &with));
  for (int i = threadIdx.x; i < kMaxSteps; i += kRowThreads) s.sums[i] = 0;
  lds_sync();
  each([&](uint64_t word, uint64_t w) {
    if (word < last) return;
    if (r.limit < kNone) w = weight(logit_of(word), r.limit);
    add64(&s.sums[index_of(word) / kStep], w);
  });
  lds_sync();
  draw_from_steps<In>(s, a, b, r, weight, last);
}

template <typename In>
__global__ __launch_bounds__(kRowThreads, 4) void row_kernel(SampleArgs a) {
  __shared__ RowShared s;
  __shared__ Powers powers;
  constexpr int kPer = Logits<In>::kPer, kLoads = kStep / kWave / kPer, kParts = kStep / kPart;
  const int64_t b = blockIdx.x / a.G;
  const int g = blockIdx.x % a.G;
  const unsigned over = a.state[b].over;
  const RowRule r = row_rule(a, b);
  if (r.kind == kGreedy && (a.top_k || a.min_p)) return;  // front_kernel's
  // A list that overflowed: under top-k one workgroup selects from the row, under min-p alone the steps are added.
  if (r.kind == kTop && (!over || (r.k && g > 0))) return;
  const uint64_t peak = row_peak(a, b);
  const float top = logit_of(peak);
  if (r.kind == kGreedy || top == -__builtin_inff()) {
    const bool open = top != -__builtin_inff();
    if (g == 0 && threadIdx.x == 0) answer(a, b, open ? index_of(peak) : -1, open ? 1.0 : 0.0);
    return;
  }
  powers.fill();
  if (threadIdx.x == 0) s.n = 0;
  lds_sync();
  const Weights weight(&powers, top, r.scale);
  if (r.kind == kTop && r.k) {
    draw_alone<In>(s, a, b, r, r.k, weight, 0);
    return;
  }

  // steps' sums; of a band's row those above what is listed
  const RowState* st = &a.state[b];
  const bool banded = r.kind == kBand && st->banded;
  const float above = st->above, reach = st->reach;
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const int end = min((g + 1) * a.chunk, a.V);
  auto all = [&](auto finite) {
    constexpr bool kFinite = decltype(finite)::value;
    auto value = [&](float l) { return weight.template operator()<kFinite>(l, r.limit); };
    float* queue = s.queue[wave];
    for (int i0 = g * a.chunk + wave * kStep; i0 < end; i0 += kRowWaves * kStep) {
      if (banded || r.limit < kNone) {  // what the step's largest logit does not reach none does
        const int i = i0 / kPart + lane;
        float most = lane < kParts && i < a.M ? a.parts[b * a.M + i] : -__builtin_inff();
        most = fmaxf(most, dpp_f32<kDppQuadXor1>(most));
        most = fmaxf(most, dpp_f32<kDppQuadXor2>(most));
        most = fmaxf(most, dpp_f32<kDppRowHalfMirror>(most));
        most = fmaxf(most, dpp_f32<kDppRowMirror>(most));
        most = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(most)));
        if (banded ? !(most >= reach) : !weight(most, r.limit)) {
          if (lane == 0) st64(&a.sums[b * kMaxSteps + i0 / kStep], 0);
          continue;
        }
      }
      Logits<In> v[kLoads];
#pragma unroll
      for (int o = 0; o < kLoads; ++o) v[o].load(row, i0 + (o * kWave + lane) * kPer, end);
      uint64_t sum = 0;
      if (!banded) {
#pragma unroll
        for (int o = 0; o < kLoads; ++o)
#pragma unroll
          for (int j = 0; j < kPer; ++j) sum += value(v[o].as_is(j));
      } else {
        // What is above goes through a queue, so that weights are computed for 64 of them at a time
        // however few they are.
        int queued = 0;
#pragma unroll
        for (int o = 0; o < kLoads; ++o) {
          bool listed = false;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const float l = v[o].as_is(j);
            const uint64_t ball = __ballot(l > above);
            listed |= l >= reach && !(l > above);
            if (ball == 0) continue;  // uniform
            if (l > above)
              queue[queued + __builtin_amdgcn_mbcnt_hi((uint32_t)(ball >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)ball, 0))] = l;
            queued += __popcll(ball);
            if (queued >= kWave) {
              __builtin_amdgcn_wave_barrier();
              const float first = queue[lane], rest = queue[lane + kWave];
              __builtin_amdgcn_wave_barrier();  // the queue is the wave's own, and LDS keeps its order
              queue[lane] = rest;
              sum += value(first);
              queued -= kWave;
            }
          }
          if (__any(listed)) {
            bool want[kPer];
            uint64_t word[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              const float l = v[o].at(j);
              want[j] = l >= reach && !(l > above) && weight.weighs(l);
              word[j] = word_of(l, i0 + (o * kWave + lane) * kPer + j);
            }
            append(s.list, &s.n, want, word);
          }
        }
        __builtin_amdgcn_wave_barrier();
        if (lane < queued) sum += value(queue[lane]);
        __builtin_amdgcn_wave_barrier();
      }
      sum = wave_sum_u64(sum);
      if (lane == 0) st64(&a.sums[b * kMaxSteps + i0 / kStep], sum);
    }
  };
  if (weight.finite()) all(std::true_type{});
  else all(std::false_type{});
  if (banded) {
    lds_sync();
    if (threadIdx.x == 0)
      s.base = s.n ? __hip_atomic_fetch_add(&a.state[b].listed, s.n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
    lds_sync();
    const unsigned base = s.base;
    for (unsigned i = threadIdx.x; i < min(s.n, (unsigned)kList) && base + i < kList; i += kRowThreads)
      st64(&a.list[b * kList + base + i], s.list[i]);
  }
  if (!last_to_arrive(&a.state[b].row_arrived, a.G)) return;

  uint64_t last = 0;
  const unsigned n = banded ? __hip_atomic_load(&a.state[b].listed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
  if (n > kList) {
    draw_alone<In>(s, a, b, r, st->k, weight, st->total);
    return;
  }
  const int steps = (a.V + kStep - 1) / kStep;
  for (int i = threadIdx.x; i < steps; i += kRowThreads) s.sums[i] = ld64(&a.sums[b * kMaxSteps + i]);
  if (banded) {
    for (unsigned i = threadIdx.x; i < n; i += kRowThreads) s.list[i] = ld64(&a.list[b * kList + i]);
    lds_sync();
    last = last_kept<kRowThreads>(s.scratch, s.list, (int)n, st->k, r.p_on, r.p, weight, Pair{st->c_base, st->w_base}, st->total);
    for (unsigned i = threadIdx.x; i < n; i += kRowThreads) {
      const uint64_t word = s.list[i], w = word >= last ? weight(logit_of(word), r.limit) : 0;
      if (w) add64(&s.sums[index_of(word) / kStep], w);
    }
  }
  lds_sync();
  draw_from_steps<In>(s, a, b, r, weight, last);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// A row's chunks: four workgroups a compute unit over all rows (256 rows of mixed parameters, few of which
// need every chunk: 103 us against 133 with two and 96 with eight), none for fewer than 4,096 tokens (37 rows of
// 32,003: 44 us against 55 with 2,048).  Taken for such mixed rows; where every row needs every chunk two
// are faster: 256 rows under a top-p of 0.9 alone 167 us against 141 with two, without a filter 75 against 71,
// 64 rows 86 against 69, and rows whose lists overflow 2.3 ms against 1.2.
void split(int64_t B, int V, int* G, int* chunk) {
  const int64_t want = std::max<int64_t>(1, 4 * (int64_t)device_cu_count() / std::max<int64_t>(B, 1));
  const int64_t n = std::max<int64_t>(1, std::min<int64_t>({want, kMaxChunks, (V + 4095) / 4096}));
  *chunk = (int)(((V + n - 1) / n + 2047) / 2048 * 2048);  // whole steps, and a peak's reads of either type
  *G = (V + *chunk - 1) / *chunk;
}

size_t carve(SampleArgs& a, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) { char* r = base ? base + off : nullptr; off += align256(bytes); return r; };
  const size_t B = (size_t)a.B;
  if (a.V <= kList) return 256;  // (not used)
  a.state = reinterpret_cast<RowState*>(take(B * sizeof(RowState)));
  a.peaks = reinterpret_cast<uint64_t*>(take(B * kMaxChunks * 8));
  a.parts = reinterpret_cast<float*>(take(B * a.M * 4));
  a.sums = reinterpret_cast<uint64_t*>(take(B * kMaxSteps * 8));
  a.list = reinterpret_cast<uint64_t*>(take(B * kList * 8));
  a.counts = reinterpret_cast<uint32_t*>(take(B * kBins * 4));
  a.weights = reinterpret_cast<uint64_t*>(take(B * kBins * 8));
  return off;
}

template <typename In>
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  const unsigned rows = (unsigned)a.B, chunks = (unsigned)(a.B * a.G);
  if (a.V <= kList) {
    hipLaunchKernelGGL(front_kernel<In>, dim3(rows), dim3(kFrontThreads), 0, stream, a, rows);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(peak_kernel<In>, dim3(chunks), dim3(kPeakThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.top_k || a.top_p || a.min_p) {
    const unsigned picks = a.top_k || a.min_p ? rows : 0;  // what a list decides
    hipLaunchKernelGGL(front_kernel<In>, dim3(picks + (a.top_k || a.top_p ? chunks : 0)), dim3(kFrontThreads), 0, stream, a, picks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(row_kernel<In>, dim3(chunks), dim3(kRowThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace_bytes(int64_t B, int V) {
  SampleArgs a{};
  a.B = B;
  a.V = V;
  a.M = (V + kPart - 1) / kPart;
  return carve(a, nullptr);
}

hipError_t run_sample(const void* logits, int is_bf16, int64_t B, int V, const float* u, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p, int32_t* ids, float* probs, void* ws,
                      hipStream_t stream) {
  SampleArgs a{};
  a.logits = logits;
  a.B = B;
  a.V = V;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.ids = ids;
  a.probs = probs;
  a.M = (V + kPart - 1) / kPart;
  split(B, V, &a.G, &a.chunk);
  carve(a, static_cast<char*>(ws));
  return is_bf16 ? launch_sample<uint16_t>(a, stream) : launch_sample<float>(a, stream);
}

}  // namespace q4moe
