// The row losses over bf16 logits (row_loss.cuh).
#include "row_loss_launch.cuh"

namespace lsdrs {
cudaError_t launch_row_loss_bf16(RowLossOp op, LossMode mode, const RowLossArgs& a,
                                 cudaStream_t s) {
  return launch_row_loss_of<RS_SCORE_BF16>(op, mode, a, s);
}
}  // namespace lsdrs
