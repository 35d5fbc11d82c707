// K-LOGPROBS over bf16 logits (logprobs.cuh).
#include "kernels.h"
#include "logprobs.cuh"

namespace lsdrs {
cudaError_t launch_logprobs_bf16(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_as<RS_SCORE_BF16>(a, s);
}
cudaError_t launch_logprobs_backward_bf16(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_backward_as<RS_SCORE_BF16>(a, s);
}
}  // namespace lsdrs
