// K-ROWLOSS: dispatch by score type (one translation unit per type, compiled
// in parallel) and the probe of its bounded wait.
#include "kernels.h"
#include "row_loss.cuh"

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

namespace {

// The ring kernel's wait on a barrier on which nothing arrives.
__global__ void row_wait_probe_kernel(uint32_t* error, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int failed;
  failed = 0;
  mbar_init(&bar, 1);
  if (wait_phase<false>(&bar, 0, &failed, limit_ns, 1000000) == kWaitRanOut) *error = kErrLookback;
}

}  // namespace

cudaError_t launch_row_wait_probe(uint32_t* error, uint64_t limit_ns, cudaStream_t s) {
  row_wait_probe_kernel<<<1, 1, 0, s>>>(error, limit_ns);
  return cudaGetLastError();
}

}  // namespace lsdrs
