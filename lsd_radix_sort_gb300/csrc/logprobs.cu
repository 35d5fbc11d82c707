// K-LOGPROBS: dispatch by score type (one translation unit per type, compiled
// in parallel).
#include "vocab.h"

#include "../../include/lsdrs.h"

namespace lsdrs {

cudaError_t launch_logprobs_f16(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_bf16(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_f32(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_backward_f16(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_backward_bf16(const LogprobArgs&, cudaStream_t);
cudaError_t launch_logprobs_backward_f32(const LogprobArgs&, cudaStream_t);

cudaError_t launch_logprobs(int type, const LogprobArgs& a, cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return launch_logprobs_f16(a, s);
    case RS_SCORE_BF16: return launch_logprobs_bf16(a, s);
    case RS_SCORE_F32: return launch_logprobs_f32(a, s);
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
