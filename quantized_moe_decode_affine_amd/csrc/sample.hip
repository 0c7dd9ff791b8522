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
// parts' maxima is a bound that at least k tokens reach, so draw_kernel, one workgroup for such a
// row, reads only the parts that reach it, lists their tokens in LDS, and finds the last
// token kept and the draw in the list.  A top-p without such a top-k needs the whole row's weights:
// band_kernel sums them by bins of max - l (bins as fine as 2^-7 of the distance) and finds
// the bin in which the filter ends; draw_kernel, on all chunks, adds up what lies above that
// bin, lists the bin, and the last workgroup of the row to arrive finds the token.  Without
// either filter draw_kernel adds up the chunks.  Where a list would overflow (many equal
// logits) the last workgroup selects from the row itself, digit by digit.
#include <algorithm>

#include "kernels.h"
#include "wave64.h"

namespace q4moe {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kPart = 64;         // tokens of a part
constexpr int kMaxChunks = 128;   // of a row
constexpr int kMaxSteps = 256;    // of a chunk: 64 * kPer tokens each
constexpr int kList = 2048;       // tokens of a row's list
constexpr int kTopMost = 1024;    // the largest top-k that goes by parts
constexpr int kBinBits = 12, kBins = 1 << kBinBits;
constexpr int kWordBits = 50, kIndexBits = 18;
constexpr uint64_t kIndexMask = (1ull << kIndexBits) - 1;
constexpr double kOne = 35184372088832.0;  // 2^45: the largest logit's weight

static_assert(kMaxSampleVocab == 1 << kIndexBits, "an index fits its bits");

// A row's state between the launches.
struct RowState {
  unsigned band_arrived, draw_arrived, listed, pad;
  unsigned expected;            // tokens in the bins that are listed
  int b_lo, b_hi;               // these bins; b_lo = kBins: none
  unsigned c_base;              // tokens in the bins before b_lo
  uint64_t w_base, total;       // their weight, and the row's
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
  uint64_t* peaks;              // [B][G] the chunk's largest word: ordered bits, index inverted
  float* parts;                 // [B][M]
  uint32_t* counts;             // [B][kBins]
  uint64_t* weights;            // [B][kBins]
  uint64_t* sums;               // [B][G]
  uint64_t* list;               // [B][kList]
  RowState* state;              // [B]
};

enum Kind { kGreedy, kAll, kTop, kBand, kSum };

struct RowRule {
  Kind kind;
  double inv_t, p, m;           // m: 0 without min-p
  int k;                        // 0 without top-k
  bool p_on;
};

__device__ __forceinline__ RowRule row_rule(const SampleArgs& a, int64_t b) {
  RowRule r;
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.0f, m = a.min_p ? a.min_p[b] : 0.0f;
  r.inv_t = 1.0 / (double)t;
  r.k = k > 0 && k < a.V ? k : 0;
  r.p_on = p < 1.0f;
  r.p = p > 0.0f ? (double)p : 0.0;
  r.m = m > 0.0f ? fmin((double)m, 1.0) : 0.0;
  r.kind = !(t > 0.0f)                                ? kGreedy
           : a.V <= kList                             ? kAll
           : r.k && r.k <= min(a.M / 2, kTopMost)     ? kTop
           : r.k || r.p_on                            ? kBand
                                                      : kSum;
  return r;
}

// A logit as the rules take it: a NaN is closed as -infinity is, and both zeros are one.
__device__ __forceinline__ float clean(float l) { return l == l ? l + 0.0f : -__builtin_inff(); }

template <typename In>
__device__ __forceinline__ float one_logit(const In* row, int i) {
  if constexpr (sizeof(In) == 2) return clean(bf16_bits_to_f32(row[i]));
  else return clean(row[i]);
}

// 16 bytes of consecutive logits from i on; closed past the row's end.
template <typename In>
struct Logits {
  static constexpr int kPer = 16 / sizeof(In);
  In raw[kPer];
  __device__ __forceinline__ void load(const In* row, int i, int V) {
    if (i + kPer <= V) {
      __builtin_memcpy(raw, row + i, 16);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if constexpr (sizeof(In) == 2) raw[j] = i + j < V ? row[i + j] : (In)0xFF80;
        else raw[j] = i + j < V ? row[i + j] : -__builtin_inff();
      }
    }
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (sizeof(In) == 2) return clean(bf16_bits_to_f32(raw[j]));
    else return clean(raw[j]);
  }
};

// The place in the order: 50 bits, larger first.
__device__ __forceinline__ uint64_t word_of(float l, int i) {
  return (uint64_t)float_key(l) << kIndexBits | (kIndexMask - (uint64_t)i);
}
__device__ __forceinline__ int index_of(uint64_t word) { return (int)(kIndexMask - (word & kIndexMask)); }
__device__ __forceinline__ float logit_of(uint64_t word) { return key_float((uint32_t)(word >> kIndexBits)); }

// Bins of the distance from the largest logit, as fine as its exponent and 7 bits from 2^-16
// to 2^16; they follow the order of the logits.
__device__ __forceinline__ int bin_of(float l, float top) {
  const float d = l == top ? 0.0f : top - l;
  constexpr int kFirst = (127 - 16) << 7;
  return min(max((int)(__float_as_uint(d) >> 16) - kFirst, 0), kBins - 1);
}

// Whether a logit has a weight at all: closed ones and those beyond 2^-46 of the largest have none, and
// change no filter's end.
__device__ __forceinline__ bool weighs(float l, float top, double inv_t) {
  return l == top || ((double)top - (double)l) * inv_t < 32.0;
}

// A token's weight; 0 where min-p drops it, and beyond 2^-46 of the largest.
__device__ __forceinline__ uint64_t weight_of(float l, float top, double inv_t, double m) {
  if (l == top) return (uint64_t)kOne;
  const double x = ((double)top - (double)l) * inv_t;
  if (!(x < 32.0)) return 0;  // closed ones among them
  const double e = exp(-x);
  if (e < m) return 0;
  // rounded to an integer by the addition: the low bits of 2^52 + v
  return (uint64_t)__double_as_longlong(e * kOne + 4503599627370496.0) & ((1ull << 52) - 1);
}

__device__ __forceinline__ uint64_t ld64(const uint64_t* p) {
  return __hip_atomic_load(const_cast<uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st64(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
// Bound by the logits' bytes.  Also clears what the row's other launches count in.
template <typename In>
__global__ __launch_bounds__(kThreads) void peak_kernel(SampleArgs a) {
  constexpr int kPer = Logits<In>::kPer, kLanes = kPart / kPer;  // lanes to a part
  constexpr int kUnroll = 4;
  __shared__ uint64_t s_best[kWaves];
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
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int o = 1; o < kWaves; ++o) w = max(w, s_best[o]);
    a.peaks[b * a.G + g] = w;
    if (g == 0) {
      RowState s{};
      s.b_lo = s.b_hi = kBins;
      a.state[b] = s;
    }
  }
  if (a.counts && row_rule(a, b).kind == kBand) {
    for (int i = g * kThreads + threadIdx.x; i < kBins; i += a.G * kThreads) {
      a.counts[b * kBins + i] = 0;
      a.weights[b * kBins + i] = 0;
    }
  }
}

// The row's largest word; every wave for itself.
__device__ __forceinline__ uint64_t row_peak(const SampleArgs& a, int64_t b) {
  uint64_t w = 0;
  for (int i = lane_id(); i < a.G; i += kWave) w = max(w, a.peaks[b * a.G + i]);
  return wave_max_u64(w);
}

// Exclusive prefix of (count, weight) over the workgroup's threads, and the totals.
struct Pair {
  uint32_t c;
  uint64_t w;
};
__device__ __forceinline__ Pair block_before(Pair mine, Pair* total) {
  __shared__ uint32_t s_c[kWaves];
  __shared__ uint64_t s_w[kWaves];
  const int wave = threadIdx.x / kWave;
  const Pair in{wave_prefix(mine.c), wave_prefix(mine.w)};
  __syncthreads();  // an earlier call's totals are read
  if (lane_id() == kWave - 1) {
    s_c[wave] = in.c;
    s_w[wave] = in.w;
  }
  __syncthreads();
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

// The least whole number that is at least p z, and 1 at least: a sum reaches p z when it
// reaches this.
__device__ __forceinline__ uint64_t share_of(double p, uint64_t z) {
  const double v = ceil(p * (double)z);
  return v < 1.0 ? 1 : min((uint64_t)v, z);
}

// ---- weights by bins, for rows whose top-p (or large top-k) ends somewhere in the row
template <typename In>
__global__ __launch_bounds__(kThreads) void band_kernel(SampleArgs a) {
  __shared__ uint64_t s_w[kBins];
  __shared__ uint32_t s_c[kBins];
  __shared__ int s_bin;
  __shared__ Pair s_before;
  constexpr int kPer = Logits<In>::kPer;
  const int64_t b = blockIdx.x / a.G;
  const int g = blockIdx.x % a.G;
  const RowRule r = row_rule(a, b);
  if (r.kind != kBand) return;
  const float top = logit_of(row_peak(a, b));
  if (top == -__builtin_inff()) return;
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s_w[i] = 0;
    s_c[i] = 0;
  }
  __syncthreads();
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  const int end = min((g + 1) * a.chunk, a.V);
  for (int i = g * a.chunk + (int)threadIdx.x * kPer; i < end; i += kThreads * kPer) {
    Logits<In> v;
    v.load(row, i, end);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float l = v.at(j);
      const uint64_t w = weight_of(l, top, r.inv_t, 0.0);
      if (w == 0) continue;  // weightless tokens change no filter's end
      const int bin = bin_of(l, top);
      atomicAdd(reinterpret_cast<unsigned long long*>(&s_w[bin]), (unsigned long long)w);
      atomicAdd(&s_c[bin], 1u);
    }
  }
  __syncthreads();
  uint32_t* counts = a.counts + b * kBins;
  uint64_t* weights = a.weights + b * kBins;
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    if (s_c[i] == 0) continue;
    __hip_atomic_fetch_add(&counts[i], s_c[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_fetch_add(&weights[i], s_w[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (!last_to_arrive(&a.state[b].band_arrived, a.G)) return;

  // the row's bins, and the ones in which the filters end
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s_c[i] = __hip_atomic_load(&counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_w[i] = ld64(&weights[i]);
  }
  __syncthreads();
  constexpr int kOwn = kBins / kThreads;
  const int own = threadIdx.x * kOwn;
  Pair mine{0, 0}, total;
  for (int i = 0; i < kOwn; ++i) {
    mine.c += s_c[own + i];
    mine.w += s_w[own + i];
  }
  const Pair before = block_before(mine, &total);
  // the first bin with which the count or the weight reaches its mark, and what lies before it
  auto find = [&](uint32_t need_c, uint64_t need_w) {
    Pair at = before;
    for (int i = 0; i < kOwn; ++i) {
      const Pair with{at.c + s_c[own + i], at.w + s_w[own + i]};
      const bool reached = need_c ? at.c < need_c && with.c >= need_c : at.w < need_w && with.w >= need_w;
      if (reached) {
        s_bin = own + i;
        s_before = at;
      }
      at = with;
    }
    __syncthreads();
  };
  RowState* st = &a.state[b];
  const bool k_on = r.k && (uint32_t)r.k <= total.c;
  int lo = kBins, hi = kBins;
  Pair base = total;
  uint64_t z = total.w;
  if (k_on) {
    find((uint32_t)r.k, 0);
    lo = hi = s_bin;
    base = s_before;
    z = base.w;  // what top-k keeps is at least that
    __syncthreads();
  }
  if (r.p_on && (!k_on || z > 0)) {
    find(0, share_of(r.p, z));
    lo = s_bin;
    base = s_before;
    if (!k_on) hi = lo;
    __syncthreads();
  } else if (r.p_on) {  // the first bin has the end of both
    lo = 0;
    base = Pair{0, 0};
  }
  Pair in{0, 0};
  for (int i = 0; i < kOwn; ++i)
    if (own + i >= lo && own + i <= hi) in.c += s_c[own + i];
  Pair listed;
  block_before(in, &listed);
  if (threadIdx.x == 0) {  // read by the next launch
    st->expected = listed.c;
    st->b_lo = lo;
    st->b_hi = hi;
    st->c_base = base.c;
    st->w_base = base.w;
    st->total = total.w;
  }
}

// ---- the draw
constexpr int kDigits = 2048;

struct DrawShared {
  uint64_t list[kList];
  union {
    struct {
      uint64_t w[kDigits];
      uint32_t c[kDigits];
    } digit;
    uint32_t bins[kBins];
    uint16_t parts[kBins];
  };
  uint64_t sums[kMaxChunks > kMaxSteps ? kMaxChunks : kMaxSteps];
  uint64_t w, word;
  uint32_t c, n;
  int at, parts_n;
};

// The word at which the count or the weight of the words from the largest on reaches its mark:
// need_c words, or need_w of weight.  each(visit) calls visit(word, weight) for this thread's share
// of the words; `bits` of them are compared, by digits of at most 11.  Returns the lowest
// word of those kept (its untold bits zero) and, in `with`, what is kept with it.
template <typename Each>
__device__ __forceinline__ uint64_t select_word(DrawShared& s, int bits, uint32_t need_c, uint64_t need_w, Each each,
                                                Pair* with) {
  uint64_t prefix = 0;
  Pair above{0, 0};
  const uint64_t mask = bits < 64 ? (1ull << bits) - 1 : ~0ull;
  int left = bits;
  while (true) {
    const int take = min(left, left > 18 ? 11 : 9);
    const int rest = left - take;
    for (int i = threadIdx.x; i < kDigits; i += kThreads) {
      s.digit.w[i] = 0;
      s.digit.c[i] = 0;
    }
    if (threadIdx.x == 0) s.at = -1;
    __syncthreads();
    each([&](uint64_t word, uint64_t w) {
      word &= mask;
      if ((left < 64 ? word >> left : 0) != prefix) return;
      const int d = (int)(word >> rest) & ((1 << take) - 1);
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.digit.w[d]), (unsigned long long)w);
      atomicAdd(&s.digit.c[d], 1u);
    });
    __syncthreads();
    // digits from the largest down, eight a thread
    constexpr int kOwn = kDigits / kThreads;
    const int own = kDigits - 1 - (int)threadIdx.x * kOwn;
    Pair mine{0, 0}, total;
    for (int i = 0; i < kOwn; ++i) {
      mine.c += s.digit.c[own - i];
      mine.w += s.digit.w[own - i];
    }
    Pair at = block_before(mine, &total);
    at.c += above.c;
    at.w += above.w;
    for (int i = 0; i < kOwn; ++i) {
      const Pair in{s.digit.c[own - i], s.digit.w[own - i]};
      const Pair up{at.c + in.c, at.w + in.w};
      // the mark is reached here, or with the last of the words where it is beyond them all
      const bool reached = need_c ? at.c < need_c && up.c >= need_c : at.w < need_w && up.w >= need_w;
      const bool end = in.c && up.c == above.c + total.c && (need_c ? up.c < need_c : up.w < need_w);
      if (reached || end) {
        s.at = own - i;
        s.c = at.c;
        s.w = at.w;
      }
      at = up;
    }
    __syncthreads();
    const int d = s.at;
    if (d < 0) {  // no word at all
      *with = above;
      __syncthreads();
      return 0;
    }
    above = Pair{s.c, s.w};
    const Pair in{s.digit.c[d], s.digit.w[d]};
    *with = Pair{above.c + in.c, above.w + in.w};
    prefix = prefix << take | (uint64_t)d;
    left = rest;
    __syncthreads();
    if (left == 0 || in.c == 1 || (need_c && with->c == need_c)) return prefix << left;
  }
}

// The first of n values (n <= 256, in LDS) with which their sum exceeds t, and the sum before it;
// every thread gets both.
__device__ __forceinline__ int first_beyond(DrawShared& s, int n, uint64_t t, uint64_t* before) {
  const int i = threadIdx.x;
  const Pair mine{0, i < n ? s.sums[i] : 0};
  Pair total;
  const Pair at = block_before(mine, &total);
  if (at.w <= t && at.w + mine.w > t) {
    s.at = i;
    s.w = at.w;
  }
  __syncthreads();
  const int found = s.at;
  *before = s.w;
  __syncthreads();
  return found;
}
static_assert(kMaxSteps <= kThreads && kMaxChunks <= kThreads, "a thread for each");

__device__ __forceinline__ uint64_t mark_of(const SampleArgs& a, int64_t b, uint64_t total) {
  const float u = a.u[b];
  const double x = u > 0.0f ? fmin((double)u, 1.0) : 0.0;
  return min((uint64_t)(x * (double)total), total - 1);
}

__device__ __forceinline__ void answer(const SampleArgs& a, int64_t b, int id, double prob) {
  a.ids[b] = id;
  if (a.probs) a.probs[b] = (float)prob;
}

// The last token that the filters keep, as its word, from a list of n words in LDS: they are all tokens
// from the one after the first base.c of the order (their weight base.w) on, down to
// the last that top-k may keep or, without top-k, to the end of the row (z = 0) or of the bin in
// which top-p ends (z: the row's weight).
__device__ __forceinline__ uint64_t last_kept(DrawShared& s, int n, const RowRule& r, float top, Pair base, uint64_t z) {
  auto each = [&](auto visit) {
    for (int i = threadIdx.x; i < n; i += kThreads) visit(s.list[i], weight_of(logit_of(s.list[i]), top, r.inv_t, 0.0));
  };
  uint64_t word = 0;
  Pair with;
  if (r.k && (uint32_t)r.k < base.c + n) {
    word = select_word(s, kWordBits, r.k - base.c, 0, each, &with);
    z = base.w + with.w;
  } else if (r.k || z == 0) {  // all of them
    Pair mine{0, 0}, total;
    each([&](uint64_t, uint64_t w) { mine.w += w; });
    block_before(mine, &total);
    z = base.w + total.w;
  }
  if (r.p_on) {
    const uint64_t need = share_of(r.p, z);
    word = max(word, select_word(s, kWordBits, 0, need > base.w ? need - base.w : 1, each, &with));
  }
  return word;
}

// The draw from a list that holds every token kept.
__device__ __forceinline__ void draw_from_list(DrawShared& s, int n, const SampleArgs& a, int64_t b, const RowRule& r,
                                               float top) {
  if (n <= kThreads) {
    // a token a thread: its place and the weight before it by comparison with all
    const int i = threadIdx.x;
    const bool here = i < n;
    const uint64_t word = here ? s.list[i] : 0;
    uint64_t w = here ? weight_of(logit_of(word), top, r.inv_t, 0.0) : 0;
    s.digit.w[i] = w;
    __syncthreads();
    uint32_t place = 0;
    uint64_t heavier = 0;
    if (r.k || r.p_on) {
      for (int j = 0; j < n; ++j) {
        const bool ahead = s.list[j] > word;
        place += ahead;
        heavier += ahead ? s.digit.w[j] : 0;
      }
    }
    bool kept = here && (!r.k || place < (uint32_t)r.k);
    Pair total;
    block_before(Pair{0, kept ? w : 0}, &total);
    if (r.p_on) kept = kept && heavier < share_of(r.p, total.w);
    if (r.m > 0.0 && kept) w = weight_of(logit_of(word), top, r.inv_t, r.m);
    if (!kept) w = 0;
    __syncthreads();
    s.digit.w[i] = w;
    block_before(Pair{0, w}, &total);
    const uint64_t t = mark_of(a, b, total.w);
    uint64_t before = 0;
    for (int j = 0; j < n; ++j) before += index_of(s.list[j]) < index_of(word) ? s.digit.w[j] : 0;
    if (here && before <= t && before + w > t) answer(a, b, index_of(word), (double)w / (double)total.w);
    return;
  }
  Pair with, total;
  const uint64_t last = last_kept(s, n, r, top, Pair{0, 0}, 0);
  auto kept = [&](uint64_t word) -> uint64_t { return word >= last ? weight_of(logit_of(word), top, r.inv_t, r.m) : 0; };
  Pair mine{0, 0};
  for (int i = threadIdx.x; i < n; i += kThreads) mine.w += kept(s.list[i]);
  block_before(mine, &total);
  // in the vocabulary's order: the inverted index from the largest down
  const uint64_t mark = mark_of(a, b, total.w) + 1;
  const uint64_t low = select_word(s, kIndexBits, 0, mark, [&](auto visit) {
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (const uint64_t w = kept(s.list[i])) visit(s.list[i], w);
  }, &with);
  // the chosen one is the kept token of the lowest inverted index from `low` on
  if (threadIdx.x == 0) s.word = kIndexMask;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t at = s.list[i] & kIndexMask;
    if (at >= low && kept(s.list[i])) atomicMin(reinterpret_cast<unsigned long long*>(&s.word), (unsigned long long)at);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if ((s.list[i] & kIndexMask) == s.word && kept(s.list[i]))
      answer(a, b, index_of(s.list[i]), (double)kept(s.list[i]) / (double)total.w);
}

// The draw from a row whose chunks' sums of kept weights are in s.sums: a kept token is one whose
// word is at least `last`.
template <typename In>
__device__ __forceinline__ void draw_from_row(DrawShared& s, const SampleArgs& a, int64_t b, const RowRule& r, float top,
                                              uint64_t last) {
  constexpr int kPer = Logits<In>::kPer, kStep = kWave * kPer;
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  const int wave = threadIdx.x / kWave, lane = lane_id();
  Pair total;
  block_before(Pair{0, (int)threadIdx.x < a.G ? s.sums[threadIdx.x] : 0}, &total);
  uint64_t t = mark_of(a, b, total.w), before;
  const int g = first_beyond(s, a.G, t, &before);
  t -= before;
  const int first = g * a.chunk, end = min(first + a.chunk, a.V), steps = (end - first + kStep - 1) / kStep;
  auto kept = [&](float l, int i) -> uint64_t {
    return word_of(l, i) >= last ? weight_of(l, top, r.inv_t, r.m) : 0;
  };
  for (int o = wave; o < steps; o += kWaves) {
    const int i = first + o * kStep + lane * kPer;
    Logits<In> v;
    v.load(row, i, end);
    uint64_t w = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) w += kept(v.at(j), i + j);
    w = wave_sum_u64(w);
    if (lane == 0) s.sums[o] = w;
  }
  __syncthreads();
  const int o = first_beyond(s, steps, t, &before);
  t -= before;
  if (wave == 0) {
    const int i = first + o * kStep + lane * kPer;
    Logits<In> v;
    v.load(row, i, end);
    uint64_t w[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) mine += w[j] = kept(v.at(j), i + j);
    uint64_t at = wave_prefix(mine) - mine;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (w[j] && at <= t && at + w[j] > t) answer(a, b, i + j, (double)w[j] / (double)total.w);
      at += w[j];
    }
  }
}

// The draw from a row by this workgroup alone: the last token kept by digits of the row's words, then
// the chunks' sums.  z: the row's weight, for a top-p without top-k.
template <typename In>
__device__ __noinline__ void draw_alone(DrawShared& s, const SampleArgs& a, int64_t b, const RowRule& r, float top,
                                        uint64_t z) {
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  auto each = [&](auto visit) {
    for (int i = threadIdx.x; i < a.V; i += kThreads) {
      const float l = one_logit(row, i);
      if (const uint64_t w = weight_of(l, top, r.inv_t, 0.0)) visit(word_of(l, i), w);
    }
  };
  uint64_t last = 0;
  Pair with;
  if (r.k) {
    last = select_word(s, kWordBits, r.k, 0, each, &with);
    z = with.w;
  }
  if (r.p_on) last = max(last, select_word(s, kWordBits, 0, share_of(r.p, z), each, &with));
  for (int g = threadIdx.x; g < a.G; g += kThreads) s.sums[g] = 0;
  __syncthreads();
  each([&](uint64_t word, uint64_t w) {
    if (word < last) return;
    if (r.m > 0.0) w = weight_of(logit_of(word), top, r.inv_t, r.m);
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.sums[index_of(word) / a.chunk]), (unsigned long long)w);
  });
  __syncthreads();
  draw_from_row<In>(s, a, b, r, top, last);
}

// Appends a wave's words to the list in LDS; false where it is full.
__device__ __forceinline__ void append(DrawShared& s, bool want, uint64_t word) {
  const uint64_t ball = __ballot(want);
  if (!ball) return;
  uint32_t base = 0;
  if (lane_id() == 0) base = atomicAdd(&s.n, (uint32_t)__popcll(ball));
  base = __builtin_amdgcn_readfirstlane(base);
  const uint32_t at = base + __popcll(ball & ((1ull << lane_id()) - 1ull));
  if (want && at < kList) s.list[at] = word;
}

template <typename In>
__global__ __launch_bounds__(kThreads) void draw_kernel(SampleArgs a) {
  __shared__ DrawShared s;
  constexpr int kPer = Logits<In>::kPer, kStep = kWave * kPer;
  const int64_t b = blockIdx.x / a.G;
  const int g = blockIdx.x % a.G;
  const RowRule r = row_rule(a, b);
  const bool alone = r.kind == kGreedy || r.kind == kAll || r.kind == kTop;
  if (alone && g > 0) return;
  const uint64_t peak = row_peak(a, b);
  const float top = logit_of(peak);
  if (r.kind == kGreedy || top == -__builtin_inff()) {
    const bool open = top != -__builtin_inff();
    if (g == 0 && threadIdx.x == 0) answer(a, b, open ? index_of(peak) : -1, open ? 1.0 : 0.0);
    return;
  }
  const In* row = static_cast<const In*>(a.logits) + b * a.V;
  const int wave = threadIdx.x / kWave, lane = lane_id();
  if (threadIdx.x == 0) {
    s.n = 0;
    s.parts_n = 0;
  }

  if (r.kind == kAll) {
    __syncthreads();
    for (int i = threadIdx.x; i - lane < a.V; i += kThreads) {
      const float l = i < a.V ? one_logit(row, i) : -__builtin_inff();
      append(s, l != -__builtin_inff(), word_of(l, i));
    }
    __syncthreads();
    draw_from_list(s, (int)s.n, a, b, r, top);
    return;
  }

  if (r.kind == kTop) {
    // the bin of the k-th largest of the parts' maxima
    constexpr int kOwnParts = kMaxSampleVocab / kPart / kThreads;
    const float* parts = a.parts + b * a.M;
    int bin[kOwnParts];
#pragma unroll
    for (int o = 0; o < kOwnParts; ++o) {
      const int i = o * kThreads + threadIdx.x;
      const float l = i < a.M ? parts[i] : -__builtin_inff();
      bin[o] = weighs(l, top, r.inv_t) ? bin_of(l, top) : kBins;
    }
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.bins[i] = 0;
    if (threadIdx.x == 0) s.at = kBins - 1;  // fewer parts than k hold a token of any weight
    __syncthreads();
#pragma unroll
    for (int o = 0; o < kOwnParts; ++o)
      if (bin[o] < kBins) atomicAdd(&s.bins[bin[o]], 1u);
    __syncthreads();
    constexpr int kOwn = kBins / kThreads;
    Pair mine{0, 0}, total;
    for (int i = 0; i < kOwn; ++i) mine.c += s.bins[threadIdx.x * kOwn + i];
    uint32_t c = block_before(mine, &total).c;
    for (int i = 0; i < kOwn; ++i) {
      const uint32_t in = s.bins[threadIdx.x * kOwn + i];
      if (c < (uint32_t)r.k && c + in >= (uint32_t)r.k) s.at = threadIdx.x * kOwn + i;
      c += in;
    }
    __syncthreads();
    const int bound = s.at;
    // the parts that reach it, then their tokens that do
#pragma unroll
    for (int o = 0; o < kOwnParts; ++o)
      if (bin[o] <= bound) s.parts[atomicAdd(&s.parts_n, 1)] = (uint16_t)(o * kThreads + threadIdx.x);
    __syncthreads();
    constexpr int kUnroll = 4;
    const int n = s.parts_n;
    for (int o = wave * kUnroll; o < n; o += kWaves * kUnroll) {
      float l[kUnroll];
      int i[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        i[j] = o + j < n ? s.parts[o + j] * kPart + lane : a.V;
        l[j] = i[j] < a.V ? one_logit(row, i[j]) : -__builtin_inff();
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        append(s, weighs(l[j], top, r.inv_t) && bin_of(l[j], top) <= bound, word_of(l[j], i[j]));
    }
    __syncthreads();
    if (s.n <= kList) draw_from_list(s, (int)s.n, a, b, r, top);
    else draw_alone<In>(s, a, b, r, top, 0);
    return;
  }

  // chunks' sums; of a band's row those above the listed bins
  const RowState st = a.state[b];
  const int b_lo = r.kind == kBand ? st.b_lo : kBins, b_hi = r.kind == kBand ? st.b_hi : kBins;
  const bool listed = b_lo < kBins && st.expected <= kList, over = b_lo < kBins && !listed;
  const int first = g * a.chunk, end = min(first + a.chunk, a.V);
  uint64_t sum = 0;
  __syncthreads();
  if (!over) {
    for (int i0 = first + wave * kStep; i0 < end; i0 += kWaves * kStep) {
      const int i = i0 + lane * kPer;
      Logits<In> v;
      v.load(row, i, end);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float l = v.at(j);
        const int bin = r.kind == kBand ? bin_of(l, top) : 0;
        if (bin < b_lo) sum += weight_of(l, top, r.inv_t, r.m);
        if (listed) append(s, bin >= b_lo && bin <= b_hi && weight_of(l, top, r.inv_t, 0.0), word_of(l, i + j));
      }
    }
  }
  sum = wave_sum_u64(sum);
  if (lane == 0) s.sums[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int o = 1; o < kWaves; ++o) sum += s.sums[o];
    st64(&a.sums[b * a.G + g], sum);
    s.c = s.n ? __hip_atomic_fetch_add(&a.state[b].listed, s.n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
  }
  __syncthreads();
  const uint32_t base = s.c;
  for (uint32_t i = threadIdx.x; i < s.n; i += kThreads) st64(&a.list[b * kList + base + i], s.list[i]);
  if (!last_to_arrive(&a.state[b].draw_arrived, a.G)) return;

  RowRule rule = r;
  if (b_lo == kBins && r.kind == kBand) rule.k = 0;  // fewer tokens have a weight than top-k keeps
  if (over) {
    if (rule.k && (uint64_t)rule.k > st.c_base + (uint64_t)st.expected) rule.k = 0;
    draw_alone<In>(s, a, b, rule, top, st.total);
    return;
  }
  uint64_t last = 0;
  if (listed) {
    const int n = (int)st.expected;
    for (int i = threadIdx.x; i < n; i += kThreads) s.list[i] = ld64(&a.list[b * kList + i]);
    if ((uint64_t)rule.k > st.c_base + (uint64_t)n) rule.k = 0;
    __syncthreads();
    last = last_kept(s, n, rule, top, Pair{st.c_base, st.w_base}, st.total);
    // that word tells the list's tokens apart, the row's others need the last one's own
    if (threadIdx.x == 0) s.word = ~0ull;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (s.list[i] >= last) atomicMin(reinterpret_cast<unsigned long long*>(&s.word), (unsigned long long)s.list[i]);
    __syncthreads();
    last = s.word;
  }
  for (int i = threadIdx.x; i < a.G; i += kThreads) s.sums[i] = ld64(&a.sums[b * a.G + i]);
  __syncthreads();
  if (listed) {
    const int n = (int)st.expected;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t word = s.list[i];
      const uint64_t w = word >= last ? weight_of(logit_of(word), top, r.inv_t, r.m) : 0;
      if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&s.sums[index_of(word) / a.chunk]), (unsigned long long)w);
    }
    __syncthreads();
  }
  draw_from_row<In>(s, a, b, rule, top, last);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// A row's chunks: about four workgroups a compute unit over all rows, none shorter than a
// workgroup's reads of two vectors a thread.
void split(int64_t B, int V, int* G, int* chunk) {
  const int64_t want = std::max<int64_t>(1, 4 * (int64_t)device_cu_count() / std::max<int64_t>(B, 1));
  int64_t n = std::min<int64_t>({want, kMaxChunks, (V + 2047) / 2048});
  n = std::max<int64_t>(n, 1);
  int64_t c = (V + n - 1) / n;
  c = (c + 2047) / 2048 * 2048;  // whole steps and parts of either type
  *chunk = (int)std::min<int64_t>(c, 65536);
  *G = (int)((V + *chunk - 1) / *chunk);
}

size_t carve(SampleArgs& a, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) { char* r = base ? base + off : nullptr; off += align256(bytes); return r; };
  const size_t B = (size_t)a.B;
  a.state = reinterpret_cast<RowState*>(take(B * sizeof(RowState)));
  a.peaks = reinterpret_cast<uint64_t*>(take(B * kMaxChunks * 8));
  a.sums = reinterpret_cast<uint64_t*>(take(B * kMaxChunks * 8));
  a.parts = reinterpret_cast<float*>(take(B * a.M * 4));
  if (a.V > kList) {
    a.list = reinterpret_cast<uint64_t*>(take(B * kList * 8));
    a.counts = reinterpret_cast<uint32_t*>(take(B * kBins * 4));
    a.weights = reinterpret_cast<uint64_t*>(take(B * kBins * 8));
  }
  return off;
}

template <typename In>
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.B * a.G)), threads(kThreads);
  hipLaunchKernelGGL(peak_kernel<In>, grid, threads, 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.V > kList && (a.top_k || a.top_p)) {
    hipLaunchKernelGGL(band_kernel<In>, grid, threads, 0, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(draw_kernel<In>, grid, threads, 0, stream, a);
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
