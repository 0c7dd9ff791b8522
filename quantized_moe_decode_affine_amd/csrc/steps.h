// Internal launchers of the operators around a layer's products: rows that are 8-bit codes
// already, the norm, microscaled 4-bit products and experts, sampling.  As in kernels.h, all
// arguments are validated before, and each returns the HIP status of its launches.
#pragma once

#include "kernels.h"

namespace q4moe {

// The same from rows that are codes [m][K] and scales [m] already; no workspace.
hipError_t run_i8_gemm_rows(const I8Mat& W, int64_t n, int K, const int8_t* codes, const float* scales, int64_t m,
                            void* Y, int out_bf16, hipStream_t stream);
hipError_t run_i8_few_rows(const I8Mat& W, int64_t n, int K, const int8_t* codes, const float* scales, int m, void* Y,
                           int out_bf16, hipStream_t stream);
// ---- root-mean-square norm (norm.hip): r, y and codes may be null
hipError_t run_rms_norm(const uint16_t* x, const uint16_t* r, const uint16_t* w, int64_t rows, int k, double eps,
                        uint16_t* total, uint16_t* y, int8_t* codes, float* scales, hipStream_t stream);

// ---- microscaled 4-bit products (mx4.hip)
struct Mx4Mat {
  const uint8_t* codes;   // [count][n][k/2]
  const uint8_t* scales;  // [count][n][k/32]
};
struct Mx4Experts {
  int hidden, inter, n_experts;
  Mx4Mat gate, up, down;           // routed, stacked by expert
  Mx4Mat sh_gate, sh_up, sh_down;  // the shared expert, or codes null
};
hipError_t run_mx4_quantize(const uint16_t* X, int64_t rows, int K, uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t run_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* Y,
                              hipStream_t stream);
size_t mx4_gemm_workspace_bytes(int64_t m, int K);
hipError_t run_mx4_gemm(const Mx4Mat& W, int64_t n, int K, const uint16_t* X, int64_t m, void* Y, int out_bf16, void* ws,
                        hipStream_t stream);
// The same for few rows, m <= 16 whose codes fit a workgroup's LDS (mx4_small.hip); no workspace.
bool mx4_few_rows(int64_t m, int K);
hipError_t run_mx4_few_rows(const Mx4Mat& W, int64_t n, int K, const uint16_t* X, int m, void* Y, int out_bf16,
                            hipStream_t stream);
// The experts on few slots (a decode step), act: mx4_few_slots_bytes of scratch.
bool mx4_few_slots(const Mx4Experts& L, int64_t T, int k);
size_t mx4_few_slots_bytes(const Mx4Experts& L, int64_t T, int k);
hipError_t run_mx4_few_slots(const Mx4Experts& L, const uint16_t* X, int T, const int32_t* ids, const float* weights,
                             int k, void* Y, int out_bf16, float* act, hipStream_t stream);
size_t experts_mx4_workspace_bytes(const Mx4Experts& L, int64_t T, int k);
hipError_t run_moe_experts_mx4(const Mx4Experts& L, const uint16_t* X, int64_t T, const int32_t* ids,
                               const float* weights, int k, void* Y, int out_bf16, void* ws, hipStream_t stream);

// ---- sampling (sample.hip): the filters' arrays and probs may be null
constexpr int kMaxSampleVocab = 1 << 18;
size_t sample_workspace_bytes(int64_t B, int V);
hipError_t run_sample(const void* logits, int is_bf16, int64_t B, int V, const float* u, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p, int32_t* ids, float* probs, void* ws,
                      hipStream_t stream);

}  // namespace q4moe
