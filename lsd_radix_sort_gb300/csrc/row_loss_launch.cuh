// Instantiations of K-ROWLOSS for one score type.
#pragma once
#include "kernels.h"
#include "row_loss.cuh"

namespace lsdrs {
template <int TYPE>
cudaError_t launch_row_loss_of(RowLossOp op, LossMode mode, const RowLossArgs& a, cudaStream_t s) {
  if (op == kOpDistill) {
    switch (mode) {
      case kLossFwd: return launch_row_loss_as<TYPE, kOpDistill, kLossFwd>(a, s);
      case kLossGrad: return launch_row_loss_as<TYPE, kOpDistill, kLossGrad>(a, s);
      case kLossBwd: return launch_row_loss_as<TYPE, kOpDistill, kLossBwd>(a, s);
    }
  } else {
    switch (mode) {
      case kLossFwd: return launch_row_loss_as<TYPE, kOpPolicy, kLossFwd>(a, s);
      case kLossGrad: return launch_row_loss_as<TYPE, kOpPolicy, kLossGrad>(a, s);
      case kLossBwd: return launch_row_loss_as<TYPE, kOpPolicy, kLossBwd>(a, s);
    }
  }
  return cudaErrorInvalidValue;
}
}  // namespace lsdrs
