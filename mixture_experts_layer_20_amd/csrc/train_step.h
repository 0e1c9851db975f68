// Launchers of routing by scores, of the products in block-scaled 8-bit floating point and of the
// AdamW step.  As those of common.h: all enqueue on `s` and return the launch status.
#pragma once

#include "common.h"

namespace moe {

// Routing by scores
struct RouteScores {
  const float* logits;   // [T, E]
  const float* bias;     // [E] or NULL
  int T, E, k, groups, topk_groups;
  bool sigmoid, renormalize;
  bool whole;            // set by the launcher
  float scale;
};
// Whether the launches fit (grids of fewer than 2^32 threads, E d an int).
bool route_scores_fits(long long T, int E);
bool route_scores_bwd_fits(long long T, long long d, int E, int k, bool dense, bool bf16);
hipError_t launch_route_scores(const RouteScores& r, int32_t* topk_idx, float* topk_gate, hipStream_t s);
// Every logit has a gradient (softmax scores that are not renormalised): dense.
inline bool route_scores_dense(bool sigmoid, bool renormalize) { return !sigmoid && !renormalize; }
size_t route_scores_bwd_ws_bytes(long long T, long long d, int E, int k, bool dense);
hipError_t launch_route_scores_bwd(const RouteScores& r, const float* dgate, const int32_t* topk_idx,
                                   const int32_t* offsets, const int32_t* src_row, const void* x, const void* w, int d,
                                   bool bf16, float* dw, void* dx, void* ws, hipStream_t s);
hipError_t launch_route_bias(const int32_t* counts, int E, float rate, const float* bias, float* out, hipStream_t s);

// Products in 8-bit floating point (E4M3) with a float scale for each block of 128
hipError_t launch_fp8_quant_rows(const void* x, long long R, int K, long long ldx, uint8_t* codes, float* scales,
                                 hipStream_t s);
hipError_t launch_fp8_quant_weights(const void* w, int G, int N, int K, uint8_t* codes, float* scales, uint8_t* codes_t,
                                    float* scales_t, hipStream_t s);
struct Fp8GemmArgs {
  const uint8_t* a;        // [M, K] codes
  const float* as;         // [K / 128, M]
  const uint8_t* b;        // [G, N, K1]
  const float* bs;         // [G, N / 128, K1 / 128]
  const uint8_t* b2;       // SwiGLU: the up rows [G, N, K]; else columns k >= ksplit, [G, N, K - ksplit]; or NULL
  const float* bs2;
  int ksplit;              // K1 = ksplit with a second source of columns, else K
  const int32_t* offsets;  // [G + 1]
  int G, M, N, K;
  void* out0;
  void* out1;
  void* out2;
  const void* aux0;
  const void* aux1;
};
hipError_t launch_fp8_gemm(int epi, const Fp8GemmArgs& a, hipStream_t s);   // epi: MxEpilogue

// AdamW over a list of tensors
struct AdamWItem {
  const void* param;
  const void* grad;
  const void* m;
  const void* v;
  const float* scale;    // 8-bit states: [2, blocks]
  const float* master;
  void* param_out;
  void* m_out;
  void* v_out;
  float* scale_out;
  float* master_out;
  long long n;
  bool bf16, grad_bf16;
  float decay;           // 1 - lr * weight decay
  uint32_t seed;
};
struct AdamWStep {
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float inv_sqrt_bc2;    // 1 / sqrt(1 - beta2^step)
  float step_size;       // lr / (1 - beta1^step)
  float eps;
  const double* sumsq;   // NULL: gradients as they are
  double max_norm;
};
hipError_t launch_adamw(const AdamWItem* items, int count, const AdamWStep& step, bool bits8, hipStream_t s);

}  // namespace moe
