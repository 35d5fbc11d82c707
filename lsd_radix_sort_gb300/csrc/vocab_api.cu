// The C ABI of a vocabulary's two ends (include/lsdrs.h): argument checks and
// launches.  Host code only; the kernels are in logprobs*.cu and embed.cu.
#include <cmath>

#include "abi_checks.h"
#include "vocab.h"

using namespace lsdrs;

namespace {

constexpr int kNameLogprobs = 10, kNameEmbed = 11;  // of the profiling log

// What both calls over rows of logits share.
rs_status logprobs_check(const rs_logprobs_args* p) {
  if (p == nullptr || !known_type(p->logits_type)) return RS_ERR_INVALID;
  const int es = score_bytes(p->logits_type);
  if (p->rows < 0 || p->rows > kMaxRows || p->cols < 1 || p->cols > RS_MAX_ROW_KEYS)
    return RS_ERR_INVALID;
  if (!matrix_ok(p->rows, p->cols, p->logits_stride, es)) return RS_ERR_INVALID;
  if (!(p->temperature >= RS_MIN_TEMPERATURE) || !std::isfinite(p->temperature))
    return RS_ERR_INVALID;
  if (p->n_tokens < 0 || p->n_tokens > RS_MAX_TOP || p->top < 0 || p->top > RS_MAX_TOP)
    return RS_ERR_INVALID;
  if (p->n_tokens > 0) {
    if (p->index_bytes != 4 && p->index_bytes != 8) return RS_ERR_INVALID;
    if (!matrix_ok(p->rows, p->n_tokens, p->tokens_stride, p->index_bytes)) return RS_ERR_INVALID;
  }
  if (p->rows == 0) return RS_OK;
  if (!given(p->logits, es) || !given(p->stats, 8)) return RS_ERR_INVALID;
  if (p->n_tokens > 0 && !given(p->tokens, p->index_bytes)) return RS_ERR_INVALID;
  return RS_OK;
}

LogprobArgs logprob_args(const rs_logprobs_args* p) {
  LogprobArgs a{};
  a.logits = p->logits;
  a.rows = p->rows;
  a.cols = p->cols;
  a.stride = p->logits_stride;
  a.tokens = p->tokens;
  a.token_stride = p->tokens_stride;
  a.index_bytes = p->index_bytes;
  a.k = p->n_tokens;
  a.top = p->top;
  a.tau = p->temperature;
  a.inv_tau = 1.0f / p->temperature;
  a.scale2 = static_cast<float>(1.4426950408889634074 / p->temperature);
  a.logprobs = p->logprobs;
  a.entropy = p->entropy;
  a.lse = p->lse;
  a.stats = reinterpret_cast<float2*>(p->stats);
  a.top_logprobs = p->top_logprobs;
  a.top_ids = p->top_ids;
  a.grad = p->grad;
  a.grad_stride = p->grad_stride;
  return a;
}

rs_status embed_grad_check(const rs_embedding_grad_args* p) {
  if (p == nullptr || !known_type(p->grad_type)) return RS_ERR_INVALID;
  if (p->out_type != p->grad_type && p->out_type != RS_SCORE_F32) return RS_ERR_INVALID;
  if (p->mode != RS_EMBED_TABLE && p->mode != RS_EMBED_ADD && p->mode != RS_EMBED_ROWS)
    return RS_ERR_INVALID;
  if (p->index_bytes != 4 && p->index_bytes != 8) return RS_ERR_INVALID;
  if (p->tokens < 0 || p->tokens > kMaxRows || p->vocab < 1 || p->vocab > kMaxRows ||
      p->width < 1 || p->width > RS_MAX_WIDTH || p->padding_id < -1 || !std::isfinite(p->scale))
    return RS_ERR_INVALID;
  const int es = score_bytes(p->grad_type), out_es = score_bytes(p->out_type);
  const bool rows = p->mode == RS_EMBED_ROWS;
  const int64_t out_rows = rows && p->tokens < p->vocab ? p->tokens : p->vocab;
  if (!matrix_ok(p->tokens, p->width, p->grad_stride, es) ||
      !matrix_ok(out_rows, p->width, p->out_stride, out_es))
    return RS_ERR_INVALID;
  if (rows && !given(p->count, 4)) return RS_ERR_INVALID;
  if (out_rows > 0 && !given(p->out, out_es)) return RS_ERR_INVALID;
  if (rows && out_rows > 0 && !given(p->row_ids, 8)) return RS_ERR_INVALID;
  if (p->tokens > 0) {
    if (!given(p->grad, es) || !given(p->ids, p->index_bytes)) return RS_ERR_INVALID;
    if (!apart(p->grad, extent(p->tokens, p->width, p->grad_stride, es), p->out,
               extent(out_rows, p->width, p->out_stride, out_es)))
      return RS_ERR_INVALID;
  }
  if (!aligned(p->status, 4)) return RS_ERR_INVALID;
  if (!given(p->temp, 256)) return RS_ERR_INVALID;
  if (p->temp_bytes < embed_grad_temp(p->tokens, p->vocab, p->width)) return RS_ERR_TEMP_TOO_SMALL;
  return RS_OK;
}

}  // namespace

extern "C" {

rs_status rs_token_logprobs_temp_bytes(int64_t rows, int64_t cols, int logits_type, int top,
                                       size_t* bytes) {
  if (!bytes || rows < 0 || rows > kMaxRows || cols < 1 || cols > RS_MAX_ROW_KEYS ||
      !known_type(logits_type) || top < 0 || top > RS_MAX_TOP)
    return RS_ERR_INVALID;
  *bytes = rows == 0 ? 0 : logprobs_temp_bytes(logits_type, rows, cols, top);
  return RS_OK;
}

rs_status rs_token_logprobs(const rs_logprobs_args* p, void* stream) {
  const rs_status st = logprobs_check(p);
  if (st != RS_OK || p->rows == 0) return st;
  if (!given(p->entropy, 4) || !given(p->lse, 4)) return RS_ERR_INVALID;
  if (p->n_tokens > 0 && !given(p->logprobs, 4)) return RS_ERR_INVALID;
  if (p->top > 0 && (!given(p->top_logprobs, 4) || !given(p->top_ids, 8))) return RS_ERR_INVALID;
  const size_t need = logprobs_temp_bytes(p->logits_type, p->rows, p->cols, p->top);
  if (!given(p->temp, 256)) return RS_ERR_INVALID;
  if (p->temp_bytes < need) return RS_ERR_TEMP_TOO_SMALL;
  LogprobArgs a = logprob_args(p);
  a.temp = p->temp;
  return enqueue(kNameLogprobs, static_cast<uint64_t>(p->rows) * p->cols, stream,
                 [&](int* n, cudaStream_t s) { return launch_logprobs(p->logits_type, a, n, s); });
}

rs_status rs_token_logprobs_backward(const rs_logprobs_args* p, const float* grad_logprobs,
                                     const float* grad_entropy, const float* grad_lse,
                                     const float* grad_top, void* stream) {
  const rs_status st = logprobs_check(p);
  if (st != RS_OK || p->rows == 0) return st;
  if (!aligned(grad_logprobs, 4) || !aligned(grad_entropy, 4) || !aligned(grad_lse, 4) ||
      !aligned(grad_top, 4))
    return RS_ERR_INVALID;
  if (grad_logprobs != nullptr && p->n_tokens == 0) return RS_ERR_INVALID;
  if (grad_top != nullptr && (p->top == 0 || !given(p->top_ids, 8))) return RS_ERR_INVALID;
  if (grad_entropy != nullptr && !given(p->entropy, 4)) return RS_ERR_INVALID;
  if (!grad_ok(p->logits, p->logits_stride, p->grad, p->grad_stride, p->rows, p->cols,
               p->logits_type))
    return RS_ERR_INVALID;
  LogprobArgs a = logprob_args(p);
  a.grad_logprobs = grad_logprobs;
  a.grad_entropy = grad_entropy;
  a.grad_lse = grad_lse;
  a.grad_top = grad_top;
  if (grad_logprobs == nullptr) a.k = 0;
  if (grad_top == nullptr) a.top = 0;
  if (grad_entropy == nullptr) a.entropy = nullptr;
  return enqueue(kNameLogprobs, static_cast<uint64_t>(p->rows) * p->cols, stream,
                 [&](int*, cudaStream_t s) {
                   return launch_logprobs_backward(p->logits_type, a, s);
                 });
}

rs_status rs_embedding(const rs_embedding_args* p, void* stream) {
  if (p == nullptr || !known_type(p->type)) return RS_ERR_INVALID;
  if (p->index_bytes != 4 && p->index_bytes != 8) return RS_ERR_INVALID;
  const int es = score_bytes(p->type);
  if (p->tokens < 0 || p->tokens > kMaxRows || p->vocab < 1 || p->vocab > kMaxRows ||
      p->width < 1 || p->width > RS_MAX_WIDTH || !std::isfinite(p->scale))
    return RS_ERR_INVALID;
  if (!matrix_ok(p->vocab, p->width, p->table_stride, es) ||
      !matrix_ok(p->tokens, p->width, p->out_stride, es))
    return RS_ERR_INVALID;
  if (!given(p->table, es)) return RS_ERR_INVALID;
  if (p->tokens == 0) return RS_OK;
  if (!given(p->ids, p->index_bytes) || !given(p->out, es)) return RS_ERR_INVALID;
  if (!apart(p->table, extent(p->vocab, p->width, p->table_stride, es), p->out,
             extent(p->tokens, p->width, p->out_stride, es)))
    return RS_ERR_INVALID;
  EmbedArgs a{};
  a.table = p->table;
  a.vocab = p->vocab;
  a.width = p->width;
  a.table_stride = p->table_stride;
  a.ids = p->ids;
  a.tokens = p->tokens;
  a.index_bytes = p->index_bytes;
  a.out = p->out;
  a.out_stride = p->out_stride;
  a.scale = p->scale;
  return enqueue(kNameEmbed, static_cast<uint64_t>(p->tokens), stream,
                 [&](int*, cudaStream_t s) { return launch_embed(p->type, a, s); });
}

rs_status rs_embedding_grad_temp_bytes(int64_t tokens, int64_t vocab, int64_t width,
                                       size_t* bytes) {
  if (!bytes || tokens < 0 || tokens > kMaxRows || vocab < 1 || vocab > kMaxRows || width < 1 ||
      width > RS_MAX_WIDTH)
    return RS_ERR_INVALID;
  *bytes = embed_grad_temp(tokens, vocab, width);
  return RS_OK;
}

rs_status rs_embedding_grad(const rs_embedding_grad_args* p, void* stream) {
  rs_status st = embed_grad_check(p);
  if (st != RS_OK) return st;
  EmbedGradArgs a{};
  a.grad = p->grad;
  a.grad_stride = p->grad_stride;
  a.tokens = p->tokens;
  a.width = p->width;
  a.vocab = p->vocab;
  a.ids = p->ids;
  a.index_bytes = p->index_bytes;
  a.padding_id = p->padding_id;
  a.scale = p->scale;
  a.mode = static_cast<EmbedGradMode>(p->mode);
  a.out = p->out;
  a.out_stride = p->out_stride;
  a.row_ids = p->row_ids;
  a.count = p->count;
  a.status = p->status;
  a.temp = p->temp;
  const uint64_t units = static_cast<uint64_t>(p->tokens);
  if (embed_grad_sorts(p->tokens)) {
    st = enqueue(kNameEmbed, units, stream,
                 [&](int*, cudaStream_t s) { return launch_embed_keys(a, s); });
    if (st == RS_OK) st = sort_embed_keys(a, stream);
    if (st != RS_OK) return st;
  }
  st = enqueue(kNameEmbed, units, stream, [&](int* n, cudaStream_t s) {
    return launch_embed_grad(p->grad_type, p->out_type, a, n, s);
  });
  return st;
}

}  // extern "C"
