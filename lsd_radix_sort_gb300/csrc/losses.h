// Launch interface between the C ABI of the losses (losses_api.cu) and their
// kernels.  Host-side structs only.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace lsdrs {

// What one call computes: the losses, the losses and the gradient, or the
// gradient from saved statistics.
enum LossMode { kLossFwd = 0, kLossGrad = 1, kLossBwd = 2 };
// Which loss is taken over the rows of logits.
enum RowLossOp { kOpDistill = 0, kOpPolicy = 1 };

struct RowLossArgs {
  const void* logits;
  int64_t rows, cols, stride;      // stride in elements
  void* grad;
  int64_t grad_stride;
  const float* weights;            // null: 1
  const float* grad_losses;        // kLossBwd; null: 1
  float* losses;
  float* lse;                      // written, or read by kLossBwd
  float inv_tau, tau;
  float scale2, scale2_low;        // log2(e) / tau: rounded, and what that leaves
  uint64_t wait_ns;                // limit on one wait of the long rows' kernel
  uint32_t* status;                // null, or set when such a wait ran out
  // distill
  const void* top_values;
  int top_type;
  int64_t top_stride;
  const void* top_indices;
  int index_bytes;
  int64_t index_stride;
  int k;
  // policy
  const void* actions;             // index_bytes each
  const float* old_logprobs;
  const float* advantages;
  const float* ref_logprobs;       // null: no KL term
  float* logprobs;
  float clip_low, clip_high, kl_coef;
};

struct BalanceArgs {
  const void* logits;
  int64_t tokens, stride;
  int experts;
  const void* ids;
  int id_bytes;
  int64_t id_stride;
  int k;
  const unsigned char* mask;       // null: every token
  float scale;
  const float* grad_loss;          // kLossBwd
  float* loss;
  int* counts;                     // written, or read by kLossBwd
  float* mean_probs;
  int* n_tokens;                   // written, or read by kLossBwd
  void* grad;
  int64_t grad_stride;
  void* temp;
};

// type: an rs_score_type
cudaError_t launch_row_loss(RowLossOp op, int type, LossMode mode, const RowLossArgs& a,
                            cudaStream_t s);
// *launched: 1, raised to the number of kernels
cudaError_t launch_balance(int type, LossMode mode, const BalanceArgs& a, int* launched,
                           cudaStream_t s);
cudaError_t launch_row_wait_probe(uint32_t* error, uint64_t limit_ns, cudaStream_t s);
// Scratch of a call; 0 where one cluster does all of it.
size_t balance_temp(int64_t tokens, int experts);

}  // namespace lsdrs
