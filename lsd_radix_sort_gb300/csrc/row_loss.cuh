// K-ROWLOSS: a loss over each row of logits and its gradient.
//
// Both losses are a function of the row's softmax statistics and of a short
// list of target columns, and both gradients have the form
//
//   grad_j = c (q_j - sum_{k: i_k = j} p_k),   q_j = exp((x_j - m) / t) / sum
//
// with the targets' probabilities p_k (distillation: the teacher's softmax
// over its list; policy: the one sampled column, p = 1) and a coefficient c
// of the row.  So one kernel serves both: a pass over the row for m and sum
// (one pass, rescaling the sum whenever the maximum grows), the coefficient,
// a pass that writes c q_j, and a last step that rewrites the target columns.
#pragma once
#include "losses.h"
#include "scores.cuh"

namespace lsdrs {

// One row's targets in shared memory (k entries each).
struct Targets {
  int* col;    // column, or -1: not live, or named before
  float* p;    // probability of the column (every entry that names it)
  float* x;    // its score
};

// What the targets contribute to the loss and the coefficient.
struct Head {
  float a;     // distill: sum p (log p - (x - ref) / t)
  float ref;   // the score that `a` is taken from: the largest target's, which
               // is near the row's maximum, so that the loss is a sum of
               // small terms instead of a difference of large ones
  int live;    // 0: the row has no target
};

template <int TYPE, int OP>
__device__ __forceinline__ void load_targets(const RowLossArgs& a, int64_t row, const Targets& t,
                                             Head* h) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  const int lane = static_cast<int>(lane_id());
  if (OP == kOpPolicy) {
    if (lane == 0) {
      const int64_t i = load_index(a.actions, a.index_bytes, row);
      const bool live = i >= 0 && i < a.cols;
      t.col[0] = live ? static_cast<int>(i) : -1;
      t.p[0] = 1.0f;
      t.x[0] = live ? S::load(x[i]) : 0.0f;
      h->live = live;
    }
    return;
  }
  const float scale2 = a.inv_tau * kLog2e;
  float vm = -INFINITY, xm = -INFINITY;
  for (int k = lane; k < a.k; k += kWarp) {
    const int64_t i = load_index(a.top_indices, a.index_bytes, row * a.index_stride + k);
    const bool live = i >= 0 && i < a.cols;
    const float v = live ? load_score(a.top_values, a.top_type, row * a.top_stride + k) : -INFINITY;
    const float xi = live ? S::load(x[i]) : -INFINITY;
    t.col[k] = live ? static_cast<int>(i) : -1;
    t.p[k] = v;
    t.x[k] = xi;
    vm = fmaxf(vm, v);
    xm = fmaxf(xm, xi);
  }
  vm = origin(warp_max(vm));
  xm = origin(warp_max(xm));
  float sum = 0.0f;
  for (int k = lane; k < a.k; k += kWarp) sum += exp2_approx((t.p[k] - vm) * scale2);
  sum = warp_sum(sum);
  const float log_sum = logf(sum);
  float acc = 0.0f;
  for (int k = lane; k < a.k; k += kWarp) {
    const float lp = (t.p[k] - vm) * a.inv_tau - log_sum;
    const float p = sum == 0.0f ? 0.0f : exp2_approx((t.p[k] - vm) * scale2) / sum;
    acc += p == 0.0f ? 0.0f : p * (lp - (t.x[k] - xm) * a.inv_tau);
    t.p[k] = p;
  }
  acc = warp_sum(acc);
  __syncwarp();
  // A column named twice: its first entry gets the sum, the others are
  // dropped.  Every lane reads before any lane writes.
  for (int k0 = 0; k0 < a.k; k0 += kWarp) {
    const int k = k0 + lane;
    const int col = k < a.k ? t.col[k] : -1;
    bool first = true;
    float p = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      if (t.col[j] == col) {
        if (j < k) first = false;
        p += t.p[j];
      }
    }
    __syncwarp();
    // entries before k0 + 32 are settled by their own group: only p changes
    if (k < a.k && first && col >= 0) t.x[k] = p;
    if (k < a.k && !first) t.x[k] = -1.0f;
    __syncwarp();
  }
  for (int k = lane; k < a.k; k += kWarp) {
    const float p = t.x[k];
    if (p < 0.0f) t.col[k] = -1;
    t.p[k] = p;
  }
  if (lane == 0) {
    h->a = acc;
    h->ref = xm;
    h->live = !(sum == 0.0f);
  }
}

// Loss, log-probability and coefficient of a row from its statistics.
struct RowResult {
  float loss, logp, lse, c;
};

template <int OP, int MODE>
__device__ __forceinline__ RowResult row_result(const RowLossArgs& a, int64_t row, float w,
                                                const Head& h, float x0, float m, float sum) {
  RowResult r;
  const bool empty = MODE == kLossBwd ? m == -INFINITY : sum == 0.0f;
  const float log_sum = MODE == kLossBwd ? 0.0f : logf(sum);
  r.lse = empty ? -INFINITY : m * a.inv_tau + log_sum;
  float up = w;
  if (MODE == kLossBwd && a.grad_losses != nullptr) up *= a.grad_losses[row];
  if (OP == kOpDistill) {
    const bool none = empty || !h.live;
    r.logp = 0.0f;
    r.loss = none ? 0.0f : a.tau * a.tau * w * (h.a + ((m - h.ref) * a.inv_tau + log_sum));
    r.c = none ? 0.0f : up * a.tau;
  } else {
    // m is the maximum, or t * lse with log_sum = 0
    const float logp = empty ? -INFINITY : (x0 - m) * a.inv_tau - log_sum;
    const float adv = a.advantages[row];
    const float ratio = expf(logp - a.old_logprobs[row]);
    const bool held = (adv > 0.0f && ratio > a.clip_high) || (adv < 0.0f && ratio < a.clip_low);
    // an advantage of 0 takes no part, however large the ratio
    const float clipped = fminf(fmaxf(ratio, a.clip_low), a.clip_high);
    float loss = adv == 0.0f ? 0.0f : -(held ? clipped : ratio) * adv;
    float g = held || adv == 0.0f ? 0.0f : -adv * ratio;
    if (isnan(ratio)) loss = g = ratio;
    if (a.ref_logprobs != nullptr) {
      const float d = a.ref_logprobs[row] - logp;
      const float e = expm1f(d);
      loss += a.kl_coef * (e - d);
      g -= a.kl_coef * e;
    }
    r.logp = logp;
    r.loss = empty ? 0.0f : w * loss;
    r.c = empty ? 0.0f : -up * g * a.inv_tau;
  }
  return r;
}

constexpr int kRowThreads = 512;

template <int TYPE, int OP, int MODE>
__global__ void __launch_bounds__(kRowThreads) row_loss_kernel(const RowLossArgs a) {
  grid_dependency_sync();
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  extern __shared__ unsigned char smem[];
  __shared__ Softmax part[kRowThreads / kWarp];
  __shared__ Head head;
  Targets t;
  t.col = reinterpret_cast<int*>(smem);
  t.p = reinterpret_cast<float*>(t.col + a.k);
  t.x = t.p + a.k;
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const float scale2 = a.inv_tau * kLog2e;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    __syncthreads();  // the last row's lists are no longer read
    const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
    Raw* g = static_cast<Raw*>(a.grad) + row * a.grad_stride;
    const float w = a.weights != nullptr ? a.weights[row] : 1.0f;
    bool off = w == 0.0f;
    if (OP == kOpPolicy) {
      const int64_t i = load_index(a.actions, a.index_bytes, row);
      off = off || i < 0 || i >= a.cols;
    }
    if (off) {
      if (MODE != kLossBwd && tid == 0) {
        a.losses[row] = 0.0f;
        a.lse[row] = 0.0f;
        if (OP == kOpPolicy) a.logprobs[row] = 0.0f;
      }
      if (MODE != kLossFwd)
        for (int64_t j = tid; j < a.cols; j += kRowThreads) g[j] = 0;
      continue;
    }
    if (warp == 0) load_targets<TYPE, OP>(a, row, t, &head);
    Softmax s{-INFINITY, 0.0f};
    if (MODE == kLossBwd) {
      s = {a.lse[row] * a.tau, 1.0f};
      __syncthreads();
    } else {
      for (int64_t j = tid; j < a.cols; j += kRowThreads) {
        const float v = S::load(x[j]);
        if (v > s.m) {
          s.sum *= exp2_approx((s.m - v) * scale2);
          s.m = v;
        }
        s.sum += exp2_approx((v - origin(s.m)) * scale2);
      }
      s = warp_join(s, scale2);
      if (lane_id() == 0) part[warp] = s;
      __syncthreads();
      s = part[0];
      for (int i = 1; i < kRowThreads / kWarp; ++i) s = join(s, part[i], scale2);
    }
    const RowResult r = row_result<OP, MODE>(a, row, w, head, t.x[0], s.m, s.sum);
    if (MODE != kLossBwd && tid == 0) {
      a.losses[row] = r.loss;
      a.lse[row] = r.lse;
      if (OP == kOpPolicy) a.logprobs[row] = r.logp;
    }
    if (MODE == kLossFwd) continue;
    const float o = origin(s.m), f = r.c / s.sum;
    auto q_of = [&](float v) { return r.c == 0.0f ? 0.0f : exp2_approx((v - o) * scale2) * f; };
    // the targets' values before any of the row is overwritten
    float fix[RS_MAX_TOP / kRowThreads];
#pragma unroll
    for (int u = 0; u < RS_MAX_TOP / kRowThreads; ++u) {
      const int k = tid + u * kRowThreads;
      if (k < a.k && t.col[k] >= 0) fix[u] = q_of(S::load(x[t.col[k]])) - r.c * t.p[k];
    }
    __syncthreads();
    for (int64_t j = tid; j < a.cols; j += kRowThreads) g[j] = S::store(q_of(S::load(x[j])));
    __syncthreads();
#pragma unroll
    for (int u = 0; u < RS_MAX_TOP / kRowThreads; ++u) {
      const int k = tid + u * kRowThreads;
      if (k < a.k && t.col[k] >= 0 && r.c != 0.0f) g[t.col[k]] = S::store(fix[u]);
    }
  }
}

template <int TYPE, int OP, int MODE>
cudaError_t launch_row_loss_as(const RowLossArgs& a, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * 4;
  const int grid = static_cast<int>(a.rows < most ? a.rows : most);
  return launch_kernel(row_loss_kernel<TYPE, OP, MODE>, dim3(grid), dim3(kRowThreads),
                       static_cast<size_t>(a.k) * 12, s, a);
}

}  // namespace lsdrs
