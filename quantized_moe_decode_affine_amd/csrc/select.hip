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

// Largest key of the wave, and the lowest lane that holds it: the maximum of the high
// words, then of the low words of the lanes that have it (12 DPP/permlane maxima instead
// of 6 64-bit compare-and-select steps of five instructions).
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t key, int* src) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  const uint32_t mh = wave_max_u32(hi);
  const uint32_t ml = wave_max_u32(hi == mh ? lo : 0u);
  *src = __builtin_ctzll(__ballot(hi == mh && lo == ml));
  return ((uint64_t)mh << 32) | ml;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

template <int V>
__global__ __launch_bounds__(kSelWaves * kWave) void select_kernel(RouteRule r, const float* __restrict__ logits,
                                                                   int64_t T, int32_t* __restrict__ ids,
                                                                   float* __restrict__ weights) {
  __shared__ double s_c[kSelWaves][V * kWave];
  const int lane = lane_id();
  const int wave = threadIdx.x / kWave;
  const int64_t t = (int64_t)blockIdx.x * kSelWaves + wave;
  if (t >= T) return;  // no workgroup barrier below: each wave works on its own row of s_c
  const float* row = logits + t * r.n_experts;
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
    l[j] = e < r.n_experts ? row[e] : -INFINITY;
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
    double* sc = s_c[wave];
#pragma unroll
    for (int j = 0; j < V; ++j) sc[lane * V + j] = c[j];
    __builtin_amdgcn_wave_barrier();
    const int per = r.n_experts / r.n_groups;
    const int shift = 31 - __builtin_clz(kWave / r.n_groups);
    const int g = lane >> shift, sub = lane & ((1 << shift) - 1);
    double t1 = -INFINITY, t2 = -INFINITY;
    if (g < r.n_groups)
      for (int j = sub; j < per; j += 1 << shift) {
        const double v = sc[g * per + j];
        t2 = fmax(t2, fmin(t1, v));
        t1 = fmax(t1, v);
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
    const float v = row[my_id];
    w = softmax ? expl(v) : sigmoid64(v);
    if (need_sum) w /= sum;
  }
  if (r.renormalise) {
    const double total = wave_sum_f64(w);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (lane < r.top_k) {
    ids[t * r.top_k + lane] = my_id;
    weights[t * r.top_k + lane] = (float)(w * (double)r.scale);
  }
}

}  // namespace

hipError_t run_select(const RouteRule& r, const float* logits, int64_t T, int32_t* ids, float* weights,
                      hipStream_t stream) {
  const dim3 grid((unsigned)((T + kSelWaves - 1) / kSelWaves)), threads(kSelWaves * kWave);
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
  float* logits = static_cast<float*>(ws);
  const hipError_t e = run_router_logits(router, r.n_experts, H, X, T, logits, stream, router_q8);
  return e != hipSuccess ? e : run_select(r, logits, T, ids, weights, stream);
}

}  // namespace q4moe
