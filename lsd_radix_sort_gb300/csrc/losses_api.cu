// The C ABI of the losses over rows of scores (include/lsdrs.h): argument
// checks and launches.  Host code only; the kernels are in row_loss*.cu and
// balance.cu.
#include <cmath>

#include "../../include/lsdrs.h"
#include "kernels.h"
#include "losses.h"

using namespace lsdrs;

namespace {

constexpr uint64_t kMaxWaitNs = 60000000000ull;
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

int score_bytes(int type) { return type == RS_SCORE_F32 ? 4 : 2; }
bool known_type(int type) { return type >= RS_SCORE_F16 && type <= RS_SCORE_F32; }
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
// a pointer that must be there, aligned to its element
bool given(const void* p, int bytes) { return p != nullptr && aligned(p, bytes); }

// rows x cols with a row stride, all addresses inside 63 bits
bool matrix_ok(int64_t rows, int64_t cols, int64_t stride, int bytes) {
  if (stride < cols) return false;
  return stride <= (int64_t(1) << 62) / bytes / (rows > 0 ? rows : 1);
}

// Bytes from the first element of a matrix to past its last.
uint64_t extent(int64_t rows, int64_t cols, int64_t stride, int bytes) {
  return rows == 0 ? 0 : (static_cast<uint64_t>(rows - 1) * stride + cols) * bytes;
}

bool apart(const void* a, uint64_t an, const void* b, uint64_t bn) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !(x < y + bn && y < x + an);
}

// The gradient lies exactly over the scores or apart from them.
bool grad_ok(const void* scores, int64_t stride, void* grad, int64_t grad_stride, int64_t rows,
             int64_t cols, int type) {
  const int es = score_bytes(type);
  if (!given(grad, es) || !matrix_ok(rows, cols, grad_stride, es)) return false;
  if (grad == scores && grad_stride == stride) return true;
  return apart(scores, extent(rows, cols, stride, es), grad,
               extent(rows, cols, grad_stride, es));
}

template <class F>
rs_status enqueue(int kernel, uint64_t units, void* stream, F&& launch) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto call = [&](int* launched) { return launch(launched, s); };
  try {
    const cudaError_t e = counted_launch(
        kernel, units, s,
        [](void* ctx, int* launched) { return (*static_cast<decltype(call)*>(ctx))(launched); },
        &call);
    return e == cudaSuccess ? RS_OK : RS_ERR_CUDA;
  } catch (...) {  // the profiling log could not grow
    return RS_ERR_CUDA;
  }
}

// What the row losses share: the logits, the row arrays, the mode's outputs.
rs_status rows_check(const void* logits, int64_t stride, int64_t rows, int64_t cols, int type,
                     const float* weights, const float* losses, const float* lse, void* grad,
                     int64_t grad_stride, float temperature, uint64_t wait_ns,
                     const uint32_t* status, LossMode mode) {
  if (!known_type(type)) return RS_ERR_INVALID;
  if (wait_ns > kMaxWaitNs || !aligned(status, 4)) return RS_ERR_INVALID;
  const int es = score_bytes(type);
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > RS_MAX_ROW_KEYS) return RS_ERR_INVALID;
  if (!matrix_ok(rows, cols, stride, es)) return RS_ERR_INVALID;
  if (!(temperature >= RS_MIN_TEMPERATURE) || !std::isfinite(temperature)) return RS_ERR_INVALID;
  if (rows == 0) return RS_OK;
  if (!given(logits, es) || !given(lse, 4) || !aligned(weights, 4)) return RS_ERR_INVALID;
  if (mode != kLossBwd && !given(losses, 4)) return RS_ERR_INVALID;
  if (mode != kLossFwd && !grad_ok(logits, stride, grad, grad_stride, rows, cols, type))
    return RS_ERR_INVALID;
  return RS_OK;
}

void set_temperature(RowLossArgs* a, float t) {
  const double scale = 1.4426950408889634074 / t;
  a->tau = t;
  a->inv_tau = 1.0f / t;
  a->scale2 = static_cast<float>(scale);
  a->scale2_low = static_cast<float>(scale - static_cast<double>(a->scale2));
}

rs_status distill(const rs_distill_args* p, const float* grad_losses, LossMode mode,
                  void* stream) {
  if (p == nullptr) return RS_ERR_INVALID;
  rs_status st = rows_check(p->logits, p->logits_stride, p->rows, p->cols, p->logits_type,
                            p->weights, p->losses, p->lse, p->grad, p->grad_stride,
                            p->temperature, p->wait_timeout_ns, p->status, mode);
  if (st != RS_OK) return st;
  if (!known_type(p->top_values_type) || p->top < 1 || p->top > RS_MAX_TOP) return RS_ERR_INVALID;
  if (p->index_bytes != 4 && p->index_bytes != 8) return RS_ERR_INVALID;
  const int ts = score_bytes(p->top_values_type);
  if (!matrix_ok(p->rows, p->top, p->top_values_stride, ts) ||
      !matrix_ok(p->rows, p->top, p->top_indices_stride, p->index_bytes))
    return RS_ERR_INVALID;
  if (p->rows == 0) return RS_OK;
  if (!given(p->top_values, ts) || !given(p->top_indices, p->index_bytes) ||
      !aligned(grad_losses, 4))
    return RS_ERR_INVALID;
  RowLossArgs a{};
  a.logits = p->logits;
  a.rows = p->rows;
  a.cols = p->cols;
  a.stride = p->logits_stride;
  a.grad = p->grad;
  a.grad_stride = p->grad_stride;
  a.weights = p->weights;
  a.grad_losses = grad_losses;
  a.losses = p->losses;
  a.lse = p->lse;
  set_temperature(&a, p->temperature);
  a.wait_ns = p->wait_timeout_ns != 0 ? p->wait_timeout_ns : kDefaultWaitNs;
  a.status = p->status;
  a.top_values = p->top_values;
  a.top_type = p->top_values_type;
  a.top_stride = p->top_values_stride;
  a.top_indices = p->top_indices;
  a.index_bytes = p->index_bytes;
  a.index_stride = p->top_indices_stride;
  a.k = p->top;
  return enqueue(8, static_cast<uint64_t>(p->rows) * p->cols, stream,
                 [&](int*, cudaStream_t s) {
                   return launch_row_loss(kOpDistill, p->logits_type, mode, a, s);
                 });
}

rs_status policy(const rs_policy_args* p, const float* grad_losses, LossMode mode, void* stream) {
  if (p == nullptr) return RS_ERR_INVALID;
  rs_status st = rows_check(p->logits, p->logits_stride, p->rows, p->cols, p->logits_type,
                            p->weights, p->losses, p->lse, p->grad, p->grad_stride,
                            p->temperature, p->wait_timeout_ns, p->status, mode);
  if (st != RS_OK) return st;
  if (p->index_bytes != 4 && p->index_bytes != 8) return RS_ERR_INVALID;
  if (!(p->clip_low >= 0.0f) || !std::isfinite(p->clip_low) || !(p->clip_high >= 0.0f) ||
      !std::isfinite(p->clip_high) || !std::isfinite(p->kl_coef))
    return RS_ERR_INVALID;
  if (p->kl_coef != 0.0f && p->rows != 0 && p->ref_logprobs == nullptr) return RS_ERR_INVALID;
  if (p->rows == 0) return RS_OK;
  if (!given(p->actions, p->index_bytes) || !given(p->old_logprobs, 4) ||
      !given(p->advantages, 4) || !aligned(p->ref_logprobs, 4) || !aligned(grad_losses, 4))
    return RS_ERR_INVALID;
  if (mode != kLossBwd && !given(p->logprobs, 4)) return RS_ERR_INVALID;
  RowLossArgs a{};
  a.logits = p->logits;
  a.rows = p->rows;
  a.cols = p->cols;
  a.stride = p->logits_stride;
  a.grad = p->grad;
  a.grad_stride = p->grad_stride;
  a.weights = p->weights;
  a.grad_losses = grad_losses;
  a.losses = p->losses;
  a.lse = p->lse;
  set_temperature(&a, p->temperature);
  a.wait_ns = p->wait_timeout_ns != 0 ? p->wait_timeout_ns : kDefaultWaitNs;
  a.status = p->status;
  a.actions = p->actions;
  a.index_bytes = p->index_bytes;
  a.k = 1;
  a.old_logprobs = p->old_logprobs;
  a.advantages = p->advantages;
  a.ref_logprobs = p->kl_coef != 0.0f ? p->ref_logprobs : nullptr;
  a.logprobs = p->logprobs;
  a.clip_low = 1.0f - p->clip_low;
  a.clip_high = 1.0f + p->clip_high;
  a.kl_coef = p->kl_coef;
  return enqueue(8, static_cast<uint64_t>(p->rows) * p->cols, stream,
                 [&](int*, cudaStream_t s) {
                   return launch_row_loss(kOpPolicy, p->logits_type, mode, a, s);
                 });
}

rs_status balance(const rs_balance_args* p, const float* grad_loss, LossMode mode, void* stream) {
  if (p == nullptr || !known_type(p->scores_type)) return RS_ERR_INVALID;
  const int es = score_bytes(p->scores_type);
  if (p->experts < 1 || p->experts > RS_MAX_EXPERTS || p->tokens < 0 || p->top < 1)
    return RS_ERR_INVALID;
  if (p->tokens > kMaxRows / p->top) return RS_ERR_INVALID;
  if (!matrix_ok(p->tokens, p->experts, p->scores_stride, es)) return RS_ERR_INVALID;
  if (!given(p->counts, 4) || !given(p->n_tokens, 4)) return RS_ERR_INVALID;
  if (mode != kLossBwd) {
    if (p->index_bytes != 4 && p->index_bytes != 8) return RS_ERR_INVALID;
    if (!matrix_ok(p->tokens, p->top, p->expert_ids_stride, p->index_bytes))
      return RS_ERR_INVALID;
    if (!given(p->loss, 4) || !given(p->mean_probs, 4)) return RS_ERR_INVALID;
    if (p->tokens > 0 && !given(p->expert_ids, p->index_bytes)) return RS_ERR_INVALID;
    const size_t need = balance_temp(p->tokens, p->experts);
    if (need != 0 && !given(p->temp, 256)) return RS_ERR_INVALID;
    if (p->temp_bytes < need) return RS_ERR_TEMP_TOO_SMALL;
    if (!std::isfinite(p->scale)) return RS_ERR_INVALID;
  }
  if (!aligned(grad_loss, 4)) return RS_ERR_INVALID;
  if (p->tokens > 0) {
    if (!given(p->scores, es)) return RS_ERR_INVALID;
    if (mode != kLossFwd && !grad_ok(p->scores, p->scores_stride, p->grad, p->grad_stride,
                                     p->tokens, p->experts, p->scores_type))
      return RS_ERR_INVALID;
  } else if (mode == kLossBwd) {
    return RS_OK;
  }
  BalanceArgs a{};
  a.logits = p->scores;
  a.tokens = p->tokens;
  a.stride = p->scores_stride;
  a.experts = p->experts;
  a.ids = p->expert_ids;
  a.id_bytes = p->index_bytes;
  a.id_stride = p->expert_ids_stride;
  a.k = p->top;
  a.mask = p->token_mask;
  a.scale = mode == kLossBwd ? 1.0f : p->scale;
  a.grad_loss = grad_loss;
  a.loss = p->loss;
  a.counts = p->counts;
  a.mean_probs = p->mean_probs;
  a.n_tokens = p->n_tokens;
  a.grad = p->grad;
  a.grad_stride = p->grad_stride;
  a.temp = p->temp;
  return enqueue(9, static_cast<uint64_t>(p->tokens), stream, [&](int* n, cudaStream_t s) {
    return launch_balance(p->scores_type, mode, a, n, s);
  });
}

}  // namespace

extern "C" {

rs_status rs_distill_loss(const rs_distill_args* args, void* stream) {
  return distill(args, nullptr, args && args->grad ? kLossGrad : kLossFwd, stream);
}

rs_status rs_distill_loss_backward(const rs_distill_args* args, const float* grad_losses,
                                   void* stream) {
  return distill(args, grad_losses, kLossBwd, stream);
}

rs_status rs_policy_loss(const rs_policy_args* args, void* stream) {
  return policy(args, nullptr, args && args->grad ? kLossGrad : kLossFwd, stream);
}

rs_status rs_policy_loss_backward(const rs_policy_args* args, const float* grad_losses,
                                  void* stream) {
  return policy(args, grad_losses, kLossBwd, stream);
}

rs_status rs_row_wait_timeout_probe(uint32_t* word, uint64_t timeout_ns, void* stream,
                                    rs_status* result) {
  if (!given(word, 4) || !result || timeout_ns == 0 || timeout_ns > kMaxWaitNs)
    return RS_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(word, 0, 4, s) != cudaSuccess) return RS_ERR_CUDA;
  const rs_status st = enqueue(4, 1, stream, [&](int*, cudaStream_t on) {
    return launch_row_wait_probe(word, timeout_ns, on);
  });
  if (st != RS_OK) return st;
  uint32_t err = 0;
  if (cudaMemcpyAsync(&err, word, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return RS_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return RS_ERR_CUDA;
  *result = static_cast<rs_status>(err);
  return RS_OK;
}

rs_status rs_balance_temp_bytes(int64_t tokens, int experts, size_t* bytes) {
  if (!bytes || tokens < 0 || tokens > kMaxRows || experts < 1 || experts > RS_MAX_EXPERTS)
    return RS_ERR_INVALID;
  *bytes = balance_temp(tokens, experts);
  return RS_OK;
}

rs_status rs_balance_loss(const rs_balance_args* args, void* stream) {
  return balance(args, nullptr, args && args->grad ? kLossGrad : kLossFwd, stream);
}

rs_status rs_balance_loss_backward(const rs_balance_args* args, const float* grad_loss,
                                   void* stream) {
  return balance(args, grad_loss, kLossBwd, stream);
}

}  // extern "C"
