// K-LOGPROBS: dispatch by score type (one translation unit per type, compiled
// in parallel).
#include "vocab.h"

#include "../../include/lsdrs.h"

namespace lsdrs {

size_t logprobs_temp_f16(int64_t, int64_t, int);
cudaError_t launch_logprobs_f16(const LogprobArgs&, int*, cudaStream_t);
size_t logprobs_temp_bf16(int64_t, int64_t, int);
cudaError_t launch_logprobs_bf16(const LogprobArgs&, int*, cudaStream_t);
size_t logprobs_temp_f32(int64_t, int64_t, int);
cudaError_t launch_logprobs_f32(const LogprobArgs&, int*, cudaStream_t);
cudaError_t launch_logprobs_backward_f16(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_backward_bf16(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_backward_f32(const LogprobArgs&, cudaStream_t);

size_t logprobs_temp_bytes(int type, int64_t rows, int64_t cols, int top) {
  switch (type) {
    case RS_SCORE_F16: return logprobs_temp_f16(rows, cols, top);
    case RS_SCORE_BF16: return logprobs_temp_bf16(rows, cols, top);
    case RS_SCORE_F32: return logprobs_temp_f32(rows, cols, top);
  }
  return 0;
}

cudaError_t launch_logprobs(int type, const LogprobArgs& a, int* launched, cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return launch_logprobs_f16(a, launched, s);
    case RS_SCORE_BF16: return launch_logprobs_bf16(a, launched, s);
    case RS_SCORE_F32: return launch_logprobs_f32(a, launched, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_logprobs_backward(int type, const LogprobArgs& a, cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return launch_logprobs_backward_f16(a, s);
    case RS_SCORE_BF16: return launch_logprobs_backward_bf16(a, s);
    case RS_SCORE_F32: return launch_logprobs_backward_f32(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lsdrs
