// K-LOGPROBS over f16 logits (logprobs.cuh).
#include "kernels.h"
#include "logprobs.cuh"

namespace lsdrs {
cudaError_t launch_logprobs_f16(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_as<RS_SCORE_F16>(a, s);
}
cudaError_t launch_logprobs_backward_f16(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_backward_as<RS_SCORE_F16>(a, s);
}
}  // namespace lsdrs
