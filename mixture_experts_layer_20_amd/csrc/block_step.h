// Launchers of the operators around the layer: the block's norms, the vocabulary loss and gradient
// clipping.  As those of common.h: all enqueue on `s` and return the launch status.
#pragma once

#include "common.h"

namespace moe {

// Norms around the block
hipError_t launch_norm_in(const void* x, const void* w, int T, int d, float eps, bool bf16, void* xn, float* rstd,
                          hipStream_t s);
// dest_pos != nullptr: y is y_perm and the combine runs in the same pass (y_out: its result, or NULL).
hipError_t launch_norm_out(const void* y, const float* topk_gate, const int32_t* dest_pos, const void* shared, int k,
                           const void* x, const void* w, const void* gate, int gate_rows, float res_scale, float eps,
                           int T, int d, bool bf16, void* y_out, void* out, float* rstd, hipStream_t s);
size_t norm_bwd_ws_bytes(long long T, int d);
hipError_t launch_norm_in_bwd(const void* dxn, const void* x, const void* w, const float* rstd, const void* dres,
                              float res_scale, int T, int d, bool bf16, void* dx, float* dw, void* ws, hipStream_t s);
hipError_t launch_norm_out_bwd(const void* dout, const void* y, const void* w, const void* gate, int gate_rows,
                               const float* rstd, int T, int d, bool bf16, void* dy, float* dw, float* dgate, void* ws,
                               hipStream_t s);

// Gradient norm and clipping
struct GradItem {
  const void* grad;
  void* out;
  long long n;
  bool bf16;
};
constexpr int kGradTable = 160;   // tensors per launch: the table stays within 4 KiB of kernel arguments
struct GradTable {
  const void* grad[kGradTable];
  void* out[kGradTable];
  int first[kGradTable + 1];     // first chunk of each tensor, among this launch's chunks
  uint32_t tail[kGradTable];     // elements of its last chunk; bit 31: bf16
  int count;
  int base;                      // chunks of the launches before this one
};
long long grad_chunks(const GradItem* g, int count);
hipError_t launch_grad_sumsq(const GradItem* g, int count, double* partial, hipStream_t s);
// sumsq, norm: either may be NULL.
hipError_t launch_grad_total(const double* partial, int count, double* sumsq, float* norm, hipStream_t s);
// sums[0..nsums): their sum is the sum of squares; nsums > 1: one more double behind them is written.
hipError_t launch_grad_scale(const GradItem* g, int count, double* sums, int nsums, float max_norm, float* norm,
                             hipStream_t s);

// Softmax cross entropy over a vocabulary
struct VocabPlan {   // moe_vocab_loss_plan_t
  int piece_words, pieces, fwd_tile, logits_tile, dh_tile, dw_tile, dh_splits, dw_splits;
};
VocabPlan vocab_loss_plan(int T, int d, int V, bool bf16);
size_t vocab_loss_ws_bytes(long long T, long long d, long long V, bool bf16);
hipError_t launch_vocab_loss(const void* h, const void* w, const int32_t* target, int T, int d, int V, bool bf16,
                             float* loss, float* lse, void* ws, hipStream_t s);
size_t vocab_loss_bwd_ws_bytes(long long T, long long d, long long V, bool bf16);
hipError_t launch_vocab_loss_bwd(const void* h, const void* w, const int32_t* target, const float* lse,
                                 const float* dloss, int T, int d, int V, bool bf16, void* dh, void* dw, void* ws,
                                 hipStream_t s);

}  // namespace moe
