// K-LOGPROBS over f32 logits (logprobs.cuh).
#include "kernels.h"
#include "logprobs.cuh"

namespace lsdrs {
size_t logprobs_temp_f32(int64_t rows, int64_t cols, int top) {
  return logprobs_temp<RS_SCORE_F32>(rows, cols, top);
}
cudaError_t launch_logprobs_f32(const LogprobArgs& a, int* launched, cudaStream_t s) {
  return launch_logprobs_as<RS_SCORE_F32>(a, launched, s);
}
cudaError_t launch_logprobs_backward_f32(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_backward_as<RS_SCORE_F32>(a, s);
}
}  // namespace lsdrs
