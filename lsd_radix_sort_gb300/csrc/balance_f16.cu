// The balance loss over f16 scores (balance.cuh).
#include "balance.cuh"

namespace lsdrs {
cudaError_t launch_balance_f16(LossMode mode, const BalanceArgs& a, int* launched, cudaStream_t s) {
  return launch_balance_of<RS_SCORE_F16>(mode, a, launched, s);
}
}  // namespace lsdrs
