// Expert selection from router logits: scores (softmax or sigmoid), a balance bias,
// groups of experts, top-k, weights (moe_route, moe_route_logits).
//
// Per token, with logits l[e] (fp32) and bias b[e]:
//   s[e] = sigmoid(l[e])  or  exp(l[e] - max l) / sum exp(l - max l)
//   c[e] = s[e] + b[e], closed where l or b is NaN or -infinity
//   group g (E/G consecutive experts): the sum of the open ones among its `terms` largest c
//   ids  = the top_k largest c of open experts in the `keep` best groups, descending
//   w    = s[ids], divided by their sum when renormalised, times `scale`
// Equal values resolve to the lower index everywhere.  Scores, choices and sums are held in
// 64 bits and each weight is rounded once to fp32: in fp32 two experts whose choices differ
// by a rounding would change places, and sigmoid would be 1 for every logit above 17.  The
// 64-bit arithmetic is a few hundred instructions a token.
//
// Measured: the selection alone 7.7 us for 2,048 tokens of 256 experts (a wave's chain of
// about 3 us after the launch; the logits are 2 MB) and 14 us for 4,093 of 512 (issue-bound:
// eight 64-bit exponentials, a sort and ten rounds a wave; the sort's conditional swaps hold a
// mask each, and at 8 and 16 experts a lane 52 and 290 of them move to lanes of vector
// registers and back).
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "topk.h"

namespace q4moe {

namespace {

constexpr int kSelWaves = 4;  // tokens per workgroup, one wave each

// Order-preserving map of a double (no NaN) to uint64; 0 is below every key.
__device__ __forceinline__ uint64_t double_key(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Largest key of the wave, and the lowest lane that holds it: the maximum of the high words,
// and only where several lanes have it (equal or nearly equal choices) that of their low words.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t key, int* src) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  const uint32_t mh = wave_max_u32(hi);
  uint64_t at = __ballot(hi == mh);
  if (at & (at - 1)) {
    const uint32_t ml = wave_max_u32(hi == mh ? lo : 0u);
    at = __ballot(hi == mh && lo == ml);
  }
  *src = __builtin_ctzll(at);
  return ((uint64_t)mh << 32) | (uint32_t)__builtin_amdgcn_readlane((int)lo, *src);
}

// Sum over the wave, by the steps of group_sum_rt on both words.
__device__ __forceinline__ double wave_sum_f64(double v) {
  auto both = [](double x, auto step) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    uint32_t a[2], b[2];
    step((uint32_t)u, a[0], b[0]);
    step((uint32_t)(u >> 32), a[1], b[1]);
    return __longlong_as_double((long long)(((uint64_t)a[1] << 32) | a[0])) +
           __longlong_as_double((long long)(((uint64_t)b[1] << 32) | b[0]));
  };
  v = both(v, [](uint32_t x, uint32_t& a, uint32_t& b) { a = x; b = dpp_u32<kDppQuadXor1>(x); });
  v = both(v, [](uint32_t x, uint32_t& a, uint32_t& b) { a = x; b = dpp_u32<kDppQuadXor2>(x); });
  v = both(v, [](uint32_t x, uint32_t& a, uint32_t& b) { a = x; b = dpp_u32<kDppRowHalfMirror>(x); });
  v = both(v, [](uint32_t x, uint32_t& a, uint32_t& b) { a = x; b = dpp_u32<kDppRowMirror>(x); });
  v = both(v, [](uint32_t x, uint32_t& a, uint32_t& b) { swap_rows16(x, a, b); });
  return both(v, [](uint32_t x, uint32_t& a, uint32_t& b) { swap_halves32(x, a, b); });
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

__device__ __forceinline__ float load_logit(const float* p, bool fresh) { return fresh ? ld_agent(p) : *p; }

// One token by one wave.  sc: V * 64 doubles of LDS of the wave's own.  kFresh: the logits
// were written by other workgroups of this launch.
template <int V, bool kFresh>
__device__ __forceinline__ void select_row(const RouteRule& r, const float* row, double* sc, int32_t* ids,
                                           float* weights) {
  const int lane = lane_id();
  const bool softmax = r.score == kScoreSoftmax;
  // the order of the choices is that of the logits unless something is added to the scores
  const bool scored = r.bias != nullptr || (r.n_groups > 1 && r.group_terms > 1);
  // a softmax score needs the row's sum unless it cancels in the renormalised weights
  const bool need_sum = softmax && (scored || !r.renormalise);

  float l[V];
  bool open[V];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    l[j] = e < r.n_experts ? load_logit(row + e, kFresh) : -INFINITY;
    open[j] = l[j] > -INFINITY;  // false for NaN
    if (open[j]) top = fmaxf(top, l[j]);
  }
  if (softmax) top = key_float(wave_max_u32(float_key(top)));
  // exp(l - max), with the maximum itself 1 (an infinite logit too) and 0 for a closed logit
  auto expl = [&](float v) -> double { return v == top ? 1.0 : v > -INFINITY ? exp((double)v - (double)top) : 0.0; };
  double sum = 0.0;
  double ex[V];
  if (need_sum) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      ex[j] = open[j] ? expl(l[j]) : 0.0;
      sum += ex[j];
    }
    sum = wave_sum_f64(sum);
  }
  double c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    if (scored) {
      const float b = r.bias && e < r.n_experts ? r.bias[e] : 0.0f;
      open[j] = open[j] && b > -INFINITY;
      c[j] = (softmax ? ex[j] / sum : sigmoid64(l[j])) + (double)b;
    } else {
      c[j] = (double)l[j] + 0.0;  // -0 becomes +0: equal logits have equal keys
    }
    if (!open[j]) c[j] = -INFINITY;
  }

  if (r.n_groups > 1) {
    // 2^shift lanes per group scan its experts, then merge their largest two
#pragma unroll
    for (int j = 0; j < V; ++j) sc[lane * V + j] = c[j];
    __builtin_amdgcn_wave_barrier();
    const int per = r.n_experts / r.n_groups;
    const int shift = 31 - __builtin_clz(kWave / r.n_groups);
    const int g = lane >> shift, sub = lane & ((1 << shift) - 1);
    double t1 = -INFINITY, t2 = -INFINITY;
    if (g < r.n_groups)
      for (int j0 = sub; j0 < per; j0 += 4 << shift) {  // four reads at a time
        double v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + (i << shift);
          v[i] = sc[g * per + min(j, per - 1)];
          if (j >= per) v[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t2 = fmax(t2, fmin(t1, v[i]));
          t1 = fmax(t1, v[i]);
        }
      }
    for (int d = 1; d < (1 << shift); d <<= 1) {
      const double o1 = __shfl_xor(t1, d, kWave), o2 = __shfl_xor(t2, d, kWave);
      t2 = fmax(fmax(t2, o2), fmin(t1, o1));
      t1 = fmax(t1, o1);
    }
    const double value = r.group_terms > 1 && t2 > -INFINITY ? t1 + t2 : t1;
    const uint64_t key = t1 > -INFINITY ? double_key(value + 0.0) : 0ull;
    int ahead = 0;
    for (int o = 0; o < r.n_groups; ++o) {
      const int from = o << shift;
      const uint64_t k2 = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), from) << 32) |
                          (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, from);
      ahead += k2 > key || (k2 == key && o < g);
    }
    if (g < r.n_groups && ahead >= r.top_groups)
      for (int j = sub; j < per; j += 1 << shift) sc[g * per + j] = -INFINITY;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = sc[lane * V + j];
  }

  // each lane's keys in descending order (stable), then top_k rounds of the largest head
  uint64_t key[V];
  int id[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    id[j] = lane * V + j;
    key[j] = c[j] > -INFINITY ? double_key(c[j]) : 0ull;
  }
#pragma unroll
  for (int a = 1; a < V; ++a)
#pragma unroll
    for (int b = a; b > 0; --b) {
      const bool sw = key[b] > key[b - 1];
      const uint64_t tk = key[b];
      const int ti = id[b];
      key[b] = sw ? key[b - 1] : key[b];
      id[b] = sw ? id[b - 1] : id[b];
      key[b - 1] = sw ? tk : key[b - 1];
      id[b - 1] = sw ? ti : id[b - 1];
    }
  int my_id = -1;
  for (int i = 0; i < r.top_k; ++i) {
    int src;
    const uint64_t m = wave_max_u64(key[0], &src);
    if (m == 0) break;  // no open expert is left: the remaining slots stay -1
    const int sel = __builtin_amdgcn_readlane(id[0], src);
    if (lane == src) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) {
        key[j] = key[j + 1];
        id[j] = id[j + 1];
      }
      key[V - 1] = 0ull;
    }
    if (lane == i) my_id = sel;
  }

  double w = 0.0;
  if (my_id >= 0) {
    const float v = load_logit(row + my_id, kFresh);
    w = softmax ? expl(v) : sigmoid64(v);
    if (need_sum) w /= sum;
  }
  if (r.renormalise) {
    const double total = wave_sum_f64(w);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (lane < r.top_k) {
    ids[lane] = my_id;
    weights[lane] = (float)(w * (double)r.scale);
  }
}

template <int V>
__global__ __launch_bounds__(kSelWaves * kWave) void select_kernel(RouteRule r, const float* __restrict__ logits,
                                                                   int64_t T, int32_t* __restrict__ ids,
                                                                   float* __restrict__ weights) {
  __shared__ double s_c[kSelWaves][V * kWave];
  const int wave = threadIdx.x / kWave;
  // no workgroup barrier below: each wave works on its own row of s_c
  for (int64_t t = (int64_t)blockIdx.x * kSelWaves + wave; t < T; t += (int64_t)gridDim.x * kSelWaves)
    select_row<V, false>(r, logits + t * r.n_experts, s_c[wave], ids + t * r.top_k, weights + t * r.top_k);
}

// Arrivals are counted in steps of an odd number (2^32 over the golden ratio), which modulo
// 2^32 has an inverse: a count that started at zero gives its workgroup's place back, and one
// that started at anything else (a workspace that was not zeroed: small integers, floats, bytes
// of ones) gives places far beyond the grid in every workgroup, but for a share of grid / 2^32
// of the values.  That costs one multiplication.
constexpr uint32_t kArrival = 0x9E3779B1u;
constexpr uint32_t inverse_u32(uint32_t a) {  // of an odd a: each step doubles the right bits, 3 at first
  uint32_t x = a;
  for (int i = 0; i < 4; ++i) x *= 2u - a * x;
  return x;
}
static_assert(kArrival * inverse_u32(kArrival) == 1u, "the inverse modulo 2^32");

// Routing of few tokens in one launch, kSelWaves of them to a group of workgroups: a wave per
// expert takes its row of the router once for the group's tokens, and the group's last
// workgroup to finish selects, a wave per token.  The launch is bound by latencies (its
// bytes, 1 MB at 256 experts of 2,048 columns, take 0.2 us): one launch instead of two saves
// one of each, 8.2 us against 12.8 for one token (and 4 us of the host's time).  `arrived`,
// a count per group, is zero before the launch and after it; where it was not, the group's
// slots get id -1 and weight NaN.
template <int V, bool kQ8>
__global__ __launch_bounds__(kSelWaves * kWave) void route_few_kernel(RouteRule r, const uint16_t* __restrict__ router,
                                                                      Q4Mat q8, int H, const uint16_t* __restrict__ X,
                                                                      int rows, float* logits, unsigned* arrived,
                                                                      int32_t* __restrict__ ids,
                                                                      float* __restrict__ weights) {
  __shared__ double s_c[kSelWaves][V * kWave];
  __shared__ uint32_t s_place;
  const int t0 = blockIdx.y * kSelWaves, T = min(kSelWaves, rows - t0);  // this group's tokens
  X += (int64_t)t0 * H;
  logits += (int64_t)t0 * r.n_experts;
  ids += t0 * r.top_k;
  weights += t0 * r.top_k;
  arrived += blockIdx.y;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int e = blockIdx.x * kSelWaves + wave;
  if (e < r.n_experts) {
    float acc[kSelWaves] = {};
    if constexpr (kQ8) {
      // 16 columns a lane and step, a quarter of a group: w = scale * q + bias
      const uint8_t* codes = reinterpret_cast<const uint8_t*>(q8.codes) + (int64_t)e * H;
      for (int j = lane * 16; j < H; j += kWave * 16) {
        const uint4 c = *reinterpret_cast<const uint4*>(codes + j);
        const float s = bf16_bits_to_f32(q8.scales[(int64_t)e * (H / kGroup) + j / kGroup]);
        const float b = bf16_bits_to_f32(q8.biases[(int64_t)e * (H / kGroup) + j / kGroup]);
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
        for (int t = 0; t < T; ++t) {
          float p = 0.f, sum = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 x = *reinterpret_cast<const uint4*>(X + (int64_t)t * H + j + 8 * h);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float lo = __uint_as_float(xw[i] << 16), hi = __uint_as_float(xw[i] & 0xFFFF0000u);
              const uint32_t w = cw[2 * h + i / 2] >> (16 * (i & 1));
              p = fmaf((float)(w & 0xFFu), lo, p);
              p = fmaf((float)((w >> 8) & 0xFFu), hi, p);
              sum += lo + hi;
            }
          }
#pragma unroll
          for (int o = 0; o < kSelWaves; ++o)
            if (o == t) acc[o] += fmaf(s, p, b * sum);
        }
      }
    } else {
      constexpr int kAhead = 4;  // pieces of 8 columns in flight per lane: 2,048 columns
      const uint16_t* w_row = router + (int64_t)e * H;
      auto dots = [&](auto tokens_c) __attribute__((always_inline)) {
        constexpr int kTokens = decltype(tokens_c)::value;  // loads of a group of fewer repeat its last
        for (int j0 = 0; j0 < H; j0 += kAhead * kWave * 8) {
          auto piece = [&](const uint16_t* row, int c) {
            const int j = j0 + (c * kWave + lane) * 8;
            return j < H ? *reinterpret_cast<const uint4*>(row + j) : make_uint4(0u, 0u, 0u, 0u);
          };
          uint4 w[kAhead], x[kTokens][kAhead];
#pragma unroll
          for (int c = 0; c < kAhead; ++c) w[c] = piece(w_row, c);
#pragma unroll
          for (int t = 0; t < kTokens; ++t)
#pragma unroll
            for (int c = 0; c < kAhead; ++c) x[t][c] = piece(X + (int64_t)min(t, T - 1) * H, c);
#pragma unroll
          for (int t = 0; t < kTokens; ++t)
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
              acc[t] = dot2_bf16(w[c].x, x[t][c].x, acc[t]);
              acc[t] = dot2_bf16(w[c].y, x[t][c].y, acc[t]);
              acc[t] = dot2_bf16(w[c].z, x[t][c].z, acc[t]);
              acc[t] = dot2_bf16(w[c].w, x[t][c].w, acc[t]);
            }
        }
      };
      if (T == 1) dots(std::integral_constant<int, 1>{});
      else dots(std::integral_constant<int, kSelWaves>{});
    }
#pragma unroll
    for (int t = 0; t < kSelWaves; ++t) {
      if (t >= T) break;
      const float l = group_sum<kWave>(acc[t]);
      if (lane == 0) st_agent(logits + (int64_t)t * r.n_experts + e, l);
    }
  }
  wait_vmem();  // this wave's logits are where every workgroup sees them
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t count = __hip_atomic_fetch_add(arrived, kArrival, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_place = count * inverse_u32(kArrival);
    if (s_place == gridDim.x - 1) __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (s_place >= gridDim.x) {  // the count did not start at zero
    for (int i = threadIdx.x; i < T * r.top_k; i += blockDim.x) {
      ids[i] = -1;
      weights[i] = __uint_as_float(0x7FC00000u);
    }
    return;
  }
  if (s_place != gridDim.x - 1 || wave >= T) return;
  select_row<V, true>(r, logits + (int64_t)wave * r.n_experts, s_c[wave], ids + wave * r.top_k,
                      weights + wave * r.top_k);
}

template <int V>
hipError_t launch_route_few(const RouteRule& r, const uint16_t* router, const Q4Mat* q8, int H, const uint16_t* X,
                            int T, float* logits, unsigned* arrived, int32_t* ids, float* weights,
                            hipStream_t stream) {
  const dim3 grid((unsigned)((r.n_experts + kSelWaves - 1) / kSelWaves), (unsigned)((T + kSelWaves - 1) / kSelWaves));
  const dim3 threads(kSelWaves * kWave);
  if (q8->codes)
    hipLaunchKernelGGL((route_few_kernel<V, true>), grid, threads, 0, stream, r, router, *q8, H, X, T, logits, arrived,
                       ids, weights);
  else
    hipLaunchKernelGGL((route_few_kernel<V, false>), grid, threads, 0, stream, r, router, *q8, H, X, T, logits,
                       arrived, ids, weights);
  return hipGetLastError();
}

// One launch where its rereading of the router by every group costs less than the second
// launch: up to 64 rows, and rows x experts up to 5,120 (16 rows of 256 experts 11.4 us against
// 13.4, 64 of 60 9.5 against 12.2; 37 of 256 18.0 against 13.7), with an 8-bit router up to
// 8,192 (16 of 256 12.1 against 17.5; 37 of 256 18.0 against 17.9).
constexpr int64_t kFewTokens = 64, kFewWork = 5120, kFewWorkQ8 = 8192;
constexpr size_t kArrivedBytes = 256;  // the groups' arrival counts, before the logits
static_assert(kFewTokens / kSelWaves * sizeof(unsigned) <= kArrivedBytes, "a count per group");

}  // namespace

size_t route_rule_workspace_bytes(int64_t T, int n_experts) {
  return kArrivedBytes + route_workspace_bytes(T, n_experts);
}

hipError_t run_select(const RouteRule& r, const float* logits, int64_t T, int32_t* ids, float* weights,
                      hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>((T + kSelWaves - 1) / kSelWaves, 1 << 20)), threads(kSelWaves * kWave);
  if (r.n_experts <= kWave)
    hipLaunchKernelGGL(select_kernel<1>, grid, threads, 0, stream, r, logits, T, ids, weights);
  else if (r.n_experts <= 4 * kWave)
    hipLaunchKernelGGL(select_kernel<4>, grid, threads, 0, stream, r, logits, T, ids, weights);
  else if (r.n_experts <= 8 * kWave)
    hipLaunchKernelGGL(select_kernel<8>, grid, threads, 0, stream, r, logits, T, ids, weights);
  else
    hipLaunchKernelGGL(select_kernel<kMaxExperts / kWave>, grid, threads, 0, stream, r, logits, T, ids, weights);
  return hipGetLastError();
}

hipError_t run_route(const RouteRule& r, const uint16_t* router, const Q4Mat* router_q8, int H, const uint16_t* X,
                     int64_t T, int32_t* ids, float* weights, void* ws, hipStream_t stream) {
  unsigned* arrived = static_cast<unsigned*>(ws);
  float* logits = reinterpret_cast<float*>(static_cast<char*>(ws) + kArrivedBytes);
  if (T <= kFewTokens && T * r.n_experts <= (router_q8->codes ? kFewWorkQ8 : kFewWork)) {
    if (r.n_experts <= kWave)
      return launch_route_few<1>(r, router, router_q8, H, X, (int)T, logits, arrived, ids, weights, stream);
    if (r.n_experts <= 4 * kWave)
      return launch_route_few<4>(r, router, router_q8, H, X, (int)T, logits, arrived, ids, weights, stream);
    if (r.n_experts <= 8 * kWave)
      return launch_route_few<8>(r, router, router_q8, H, X, (int)T, logits, arrived, ids, weights, stream);
    return launch_route_few<kMaxExperts / kWave>(r, router, router_q8, H, X, (int)T, logits, arrived, ids, weights,
                                                 stream);
  }
  const hipError_t e = run_router_logits(router, r.n_experts, H, X, T, logits, stream, router_q8);
  return e != hipSuccess ? e : run_select(r, logits, T, ids, weights, stream);
}

}  // namespace q4moe
