// K-ROWLOSS dispatch by score type; one translation unit per type, compiled
// in parallel.
#include "kernels.h"
#include "losses.h"
#include "../../include/lsdrs.h"

namespace lsdrs {

cudaError_t launch_row_loss_f16(RowLossOp, LossMode, const RowLossArgs&, cudaStream_t);
cudaError_t launch_row_loss_bf16(RowLossOp, LossMode, const RowLossArgs&, cudaStream_t);
cudaError_t launch_row_loss_f32(RowLossOp, LossMode, const RowLossArgs&, cudaStream_t);

cudaError_t launch_row_loss(RowLossOp op, int type, LossMode mode, const RowLossArgs& a,
                            cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return launch_row_loss_f16(op, mode, a, s);
    case RS_SCORE_BF16: return launch_row_loss_bf16(op, mode, a, s);
    case RS_SCORE_F32: return launch_row_loss_f32(op, mode, a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lsdrs
