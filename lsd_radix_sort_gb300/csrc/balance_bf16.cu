// The balance loss over bf16 scores (balance.cuh).
#include "balance.cuh"

namespace lsdrs {
cudaError_t launch_balance_bf16(LossMode mode, const BalanceArgs& a, int* launched,
                                cudaStream_t s) {
  return launch_balance_of<RS_SCORE_BF16>(mode, a, launched, s);
}
}  // namespace lsdrs
