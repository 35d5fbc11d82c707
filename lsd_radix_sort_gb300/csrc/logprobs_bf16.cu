// K-LOGPROBS over bf16 logits (logprobs.cuh).
#include "kernels.h"
#include "logprobs.cuh"

namespace lsdrs {
size_t logprobs_temp_bf16(int64_t rows, int64_t cols, int top) {
  return logprobs_temp<RS_SCORE_BF16>(rows, cols, top);
}
cudaError_t launch_logprobs_bf16(const LogprobArgs& a, int* launched, cudaStream_t s) {
  return launch_logprobs_as<RS_SCORE_BF16>(a, launched, s);
}
cudaError_t launch_logprobs_backward_bf16(const LogprobArgs& a, cudaStream_t s) {
  return launch_logprobs_backward_as<RS_SCORE_BF16>(a, s);
}
}  // namespace lsdrs
