// Launch interface between the C ABI of the vocabulary's two ends
// (vocab_api.cu) and their kernels.  Host-side structs only.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/lsdrs.h"

namespace lsdrs {

struct LogprobArgs {
  const void* logits;
  int64_t rows, cols, stride;      // stride in elements
  const void* tokens;              // k per row, index_bytes each
  int64_t token_stride;
  int index_bytes, k, top;
  float tau, inv_tau, scale2;      // scale2 = log2(e) / tau
  float* logprobs;
  float* entropy;                  // written, or read by the backward call
  float* lse;
  float2* stats;                   // a row's largest score and log-sum; likewise
  float* top_logprobs;
  int64_t* top_ids;                // likewise
  void* temp;                      // of the forward call
  // the backward call; each upstream gradient may be null
  const float* grad_logprobs;
  const float* grad_entropy;
  const float* grad_lse;
  const float* grad_top;
  void* grad;
  int64_t grad_stride;
};

struct EmbedArgs {
  const void* table;
  int64_t vocab, width, table_stride;  // strides in elements
  const void* ids;
  int64_t tokens;
  int index_bytes;
  void* out;
  int64_t out_stride;
  float scale;
};

// Where the gradient of an embedding goes.
enum EmbedGradMode { kEmbedTable = 0, kEmbedAdd = 1, kEmbedRows = 2 };

struct EmbedGradArgs {
  const void* grad;                // tokens x width
  int64_t grad_stride, tokens, width, vocab;
  const void* ids;
  int index_bytes;
  int64_t padding_id;              // this id gets no gradient (-1: none does not)
  float scale;
  EmbedGradMode mode;
  void* out;                       // vocab rows, or min(tokens, vocab) (kEmbedRows)
  int64_t out_stride;
  int64_t* row_ids;                // kEmbedRows
  int* count;                      // kEmbedRows
  uint32_t* status;                // null, or set when a wait of the sort ran out
  void* temp;
};

// type: an rs_score_type
// Scratch of a forward call.
size_t logprobs_temp_bytes(int type, int64_t rows, int64_t cols, int top);
cudaError_t launch_logprobs(int type, const LogprobArgs& a, int* launched, cudaStream_t s);
cudaError_t launch_logprobs_backward(int type, const LogprobArgs& a, cudaStream_t s);
cudaError_t launch_embed(int type, const EmbedArgs& a, cudaStream_t s);
// The gradient: its launches, after those of a sort of whole keys where there
// are too many tokens for less.  out_type: the input's, or RS_SCORE_F32.
size_t embed_grad_temp(int64_t tokens, int64_t vocab, int64_t width);
bool embed_grad_sorts(int64_t tokens);
cudaError_t launch_embed_keys(const EmbedGradArgs& a, cudaStream_t s);
rs_status sort_embed_keys(const EmbedGradArgs& a, void* stream);
cudaError_t launch_embed_grad(int type, int out_type, const EmbedGradArgs& a, int* launched,
                              cudaStream_t s);

}  // namespace lsdrs
