// K-LOGPROBS over f32 logits (logprobs.cuh).
#include "kernels.h"
#include "logprobs.cuh"

namespace lsdrs {
cudaError_t launch_logprobs_f32(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_as<RS_SCORE_F32>(a, s);
}
cudaError_t launch_logprobs_backward_f32(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_backward_as<RS_SCORE_F32>(a, s);
}
}  // namespace lsdrs
