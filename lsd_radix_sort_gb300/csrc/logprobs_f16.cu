// K-LOGPROBS over f16 logits (logprobs.cuh).
#include "kernels.h"
#include "logprobs.cuh"

namespace lsdrs {
size_t logprobs_temp_f16(int64_t rows, int64_t cols, int top) {
  return logprobs_temp<RS_SCORE_F16>(rows, cols, top);
}
cudaError_t launch_logprobs_f16(const LogprobArgs& a, int* launched, cudaStream_t s) {
  return launch_logprobs_as<RS_SCORE_F16>(a, launched, s);
}
cudaError_t launch_logprobs_backward_f16(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_backward_as<RS_SCORE_F16>(a, s);
}
}  // namespace lsdrs
