// The balance loss over f32 scores (balance.cuh).
#include "balance.cuh"

namespace lsdrs {
cudaError_t launch_balance_f32(LossMode mode, const BalanceArgs& a, int* launched, cudaStream_t s) {
  return launch_balance_of<RS_SCORE_F32>(mode, a, launched, s);
}
}  // namespace lsdrs
