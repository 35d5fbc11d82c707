// K-BALANCE: a router's load-balancing loss, its per-expert counts and the
// gradient.
//
// With p = softmax of a token's scores and c the counts of the expert ids,
// loss = E / (K N^2) sum_e c_e sum_t p_te and
// d loss / d x_tj = E / (K N^2) p_tj (c_j - sum_e c_e p_te): the gradient
// needs the counts of all tokens, but not the probabilities' sums.  So the
// ids (a few words per token) are counted first; then one pass reads each
// token's scores once, adds its probabilities to per-lane sums (a lane always
// holds the same experts) and writes its gradient.
#include "kernels.h"
#include "losses.h"
#include "scores.cuh"

namespace lsdrs {

namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / kWarp;

// Scratch: one ticket, then one row of experts floats per CTA.
constexpr int kBalMaxCtas = 304;
constexpr size_t kBalHeader = 256;

__global__ void __launch_bounds__(kBalThreads) balance_zero_kernel(const BalanceArgs a) {
  grid_dependency_sync();
  for (int e = threadIdx.x; e < a.experts; e += kBalThreads) a.counts[e] = 0;
  if (threadIdx.x == 0) {
    *a.n_tokens = 0;
    *static_cast<unsigned*>(a.temp) = 0;
  }
}

__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(const BalanceArgs a) {
  grid_dependency_sync();
  __shared__ int hist[RS_MAX_EXPERTS + 1];
  for (int e = threadIdx.x; e <= a.experts; e += kBalThreads) hist[e] = 0;
  __syncthreads();
  const int64_t n = a.tokens * a.k;
  for (int64_t i = blockIdx.x * int64_t(kBalThreads) + threadIdx.x; i < n;
       i += int64_t(gridDim.x) * kBalThreads) {
    const int64_t t = i / a.k;
    const int s = static_cast<int>(i - t * a.k);
    if (a.mask != nullptr && !a.mask[t]) continue;
    const int64_t e = load_index(a.ids, a.id_bytes, t * a.id_stride + s);
    if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
    if (s == 0) atomicAdd(&hist[a.experts], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.experts; e += kBalThreads)
    if (hist[e] != 0) atomicAdd(e < a.experts ? a.counts + e : a.n_tokens, hist[e]);
}

template <int TYPE, int MODE, int COLS>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(const BalanceArgs a) {
  grid_dependency_sync();
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  __shared__ float share[RS_MAX_EXPERTS];  // E c_e / (K N)
  __shared__ float sums[MODE == kLossBwd ? 1 : RS_MAX_EXPERTS];
  __shared__ bool last;
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  const float n = fmaxf(static_cast<float>(*a.n_tokens), 1.0f);
  for (int e = tid; e < a.experts; e += kBalThreads)
    share[e] = static_cast<float>(a.counts[e]) * a.experts / (a.k * n);
  __syncthreads();
  float scale = a.scale;
  if (MODE == kLossBwd && a.grad_loss != nullptr) scale *= *a.grad_loss;
  scale /= n;
  float acc[COLS];
#pragma unroll
  for (int u = 0; u < COLS; ++u) acc[u] = 0.0f;
  for (int64_t t = blockIdx.x * int64_t(kBalWarps) + tid / kWarp; t < a.tokens;
       t += int64_t(gridDim.x) * kBalWarps) {
    Raw* g = static_cast<Raw*>(a.grad) + t * a.grad_stride;
    if (a.mask != nullptr && !a.mask[t]) {
      if (MODE != kLossFwd)
        for (int e = lane; e < a.experts; e += kWarp) g[e] = 0;
      continue;
    }
    const Raw* x = static_cast<const Raw*>(a.logits) + t * a.stride;
    float v[COLS], m = -INFINITY;
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
      const int e = u * kWarp + lane;
      v[u] = e < a.experts ? S::load(x[e]) : -INFINITY;
      m = fmaxf(m, v[u]);
    }
    m = origin(warp_max(m));
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
      const int e = u * kWarp + lane;
      v[u] = exp2_approx((v[u] - m) * kLog2e);
      sum += v[u];
      if (MODE != kLossFwd && e < a.experts) dot += v[u] * share[e];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (MODE != kLossFwd) dot = warp_sum(dot) * inv;
#pragma unroll
    for (int u = 0; u < COLS; ++u) {
      const int e = u * kWarp + lane;
      const float p = v[u] * inv;
      acc[u] += p;
      if (MODE != kLossFwd && e < a.experts) g[e] = S::store(p * (share[e] - dot) * scale);
    }
  }
  if (MODE == kLossBwd) return;
  // per-warp sums, added in warp order, then per-CTA sums in CTA order by the
  // CTA that finishes last: the same bits in every run
  for (int e = tid; e < a.experts; e += kBalThreads) sums[e] = 0.0f;
  for (int wp = 0; wp < kBalWarps; ++wp) {
    __syncthreads();
    if (tid / kWarp == wp) {
#pragma unroll
      for (int u = 0; u < COLS; ++u)
        if (u * kWarp + lane < a.experts) sums[u * kWarp + lane] += acc[u];
    }
  }
  __syncthreads();
  float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.temp) + kBalHeader);
  for (int e = tid; e < a.experts; e += kBalThreads)
    part[static_cast<size_t>(blockIdx.x) * a.experts + e] = sums[e];
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(static_cast<unsigned*>(a.temp), 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float loss = 0.0f;
  for (int e = tid; e < a.experts; e += kBalThreads) {
    float p = 0.0f;
    for (unsigned b = 0; b < gridDim.x; ++b) p += __ldcg(part + static_cast<size_t>(b) * a.experts + e);
    p /= n;
    a.mean_probs[e] = p;
    loss += share[e] * p;
  }
  loss = warp_sum(loss);
  __syncthreads();
  if (lane == 0) sums[tid / kWarp] = loss;
  __syncthreads();
  if (tid == 0) {
    loss = 0.0f;
    for (int i = 0; i < kBalWarps; ++i) loss += sums[i];
    *a.loss = loss;
  }
}

template <int TYPE, int MODE>
cudaError_t launch_cols(const BalanceArgs& a, int* launched, cudaStream_t s) {
  if (MODE != kLossBwd) {
    cudaError_t e = launch_kernel(balance_zero_kernel, dim3(1), dim3(kBalThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.tokens * a.k + kBalThreads - 1) / kBalThreads;
    const int grid = static_cast<int>(want < 1 ? 1 : want < kBalMaxCtas ? want : kBalMaxCtas);
    e = launch_kernel(balance_count_kernel, dim3(grid), dim3(kBalThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    *launched = 3;
  }
  const int64_t want = (a.tokens + kBalWarps - 1) / kBalWarps;
  const int grid = static_cast<int>(want < 1 ? 1 : want < kBalMaxCtas ? want : kBalMaxCtas);
  const int cols = (a.experts + kWarp - 1) / kWarp;
  auto go = [&](auto kern) { return launch_kernel(kern, dim3(grid), dim3(kBalThreads), 0, s, a); };
  if (cols <= 1) return go(balance_kernel<TYPE, MODE, 1>);
  if (cols <= 2) return go(balance_kernel<TYPE, MODE, 2>);
  if (cols <= 4) return go(balance_kernel<TYPE, MODE, 4>);
  if (cols <= 8) return go(balance_kernel<TYPE, MODE, 8>);
  if (cols <= 16) return go(balance_kernel<TYPE, MODE, 16>);
  return go(balance_kernel<TYPE, MODE, 32>);
}

template <int TYPE>
cudaError_t launch_mode(LossMode mode, const BalanceArgs& a, int* launched, cudaStream_t s) {
  switch (mode) {
    case kLossFwd: return launch_cols<TYPE, kLossFwd>(a, launched, s);
    case kLossGrad: return launch_cols<TYPE, kLossGrad>(a, launched, s);
    case kLossBwd: return launch_cols<TYPE, kLossBwd>(a, launched, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t balance_temp(int experts) {
  return kBalHeader + align_up(static_cast<size_t>(kBalMaxCtas) * experts * sizeof(float), 256);
}

cudaError_t launch_balance(int type, LossMode mode, const BalanceArgs& a, int* launched,
                           cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return launch_mode<RS_SCORE_F16>(mode, a, launched, s);
    case RS_SCORE_BF16: return launch_mode<RS_SCORE_BF16>(mode, a, launched, s);
    case RS_SCORE_F32: return launch_mode<RS_SCORE_F32>(mode, a, launched, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lsdrs
