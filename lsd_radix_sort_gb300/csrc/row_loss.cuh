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
#include <atomic>
#include <climits>

#include "losses.h"
#include "scores.cuh"

namespace lsdrs {

// One row's targets in shared memory (k entries each).
struct Targets {
  int* col;    // column, or -1: not live, or named before
  float* p;    // probability of the column (every entry that names it)
  float* x;    // its score
};

// A distillation loss is added up in units of scores, a 64th of it at a time: a
// target masked by the type's lowest value is twice that from the largest score
// there may be, more than a float holds, and so is the lowest value over a
// temperature below 1, or 21 temperatures (the logarithm of 2^30 columns) near
// a float's end; weight and temperature come last.
constexpr float kPart = 1.0f / 64;

// What the target warp hands to the threads that hold the row.
struct Head {
  int off;       // weight 0 (or no action): the row is not read
  int live;      // 0: the row has no target
  float w, up;   // weight; weight times the upstream gradient
  float a;       // distill: t sum p (log p - (x - ref) / t), kPart of it
  float ref;     // the score that `a` is taken from: the largest target's,
                 // which is near the row's maximum, so that the loss is a sum
                 // of small terms instead of a difference of large ones
  float x0, adv, old, ref_logp;  // policy
};

// Slots of the table in which the columns of k entries are looked up: a power
// of two, at least 2 k.
__host__ __device__ constexpr inline int target_slots(int k) {
  int n = 64;
  while (n < 2 * k) n *= 2;
  return n;
}

// Whether the row takes part at all; read by every warp that decides on it.
template <int OP>
__device__ __forceinline__ bool row_off(const RowLossArgs& a, int64_t row) {
  bool off = a.weights != nullptr && a.weights[row] == 0.0f;
  if (OP == kOpPolicy) {
    const int64_t i = load_index(a.actions, a.index_bytes, row);
    off = off || i < 0 || i >= a.cols;
  }
  return off;
}

// One warp reads a row's targets: their columns, scores and probabilities,
// and what they contribute to the loss.  slots: target_slots(k) words.
template <int TYPE, int OP, int MODE>
__device__ __forceinline__ void load_targets(const RowLossArgs& a, int64_t row, const Targets& t,
                                             int* slots, Head* h) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  const int lane = static_cast<int>(lane_id());
  const float w = a.weights != nullptr ? a.weights[row] : 1.0f;
  const float up = MODE == kLossBwd && a.grad_losses != nullptr ? w * a.grad_losses[row] : w;
  if (OP == kOpPolicy) {
    if (lane == 0) {
      const int64_t i = load_index(a.actions, a.index_bytes, row);
      const bool live = i >= 0 && i < a.cols;
      t.col[0] = live ? static_cast<int>(i) : -1;
      t.p[0] = 1.0f;
      const float x0 = live ? S::load(x[i]) : 0.0f;
      t.x[0] = x0;
      h->off = !live || w == 0.0f;
      h->live = 1;
      h->w = w;
      h->up = up;
      h->x0 = x0;
      h->adv = a.advantages[row];
      h->old = a.old_logprobs[row];
      h->ref_logp = a.ref_logprobs != nullptr ? a.ref_logprobs[row] : 0.0f;
    }
    return;
  }
  if (w == 0.0f) {  // neither the list nor the row is read
    if (lane == 0) h->off = 1;
    return;
  }
  const float scale2 = a.scale2;
  float vm = -INFINITY, xm = -INFINITY;
  // Columns and values of up to 256 entries are in flight together, then
  // their scores: two trips to memory, whatever the length up to there.
  constexpr int kBatch = 8;
  for (int k0 = lane; k0 < a.k; k0 += kBatch * kWarp) {
    int col[kBatch];
    float v[kBatch], xi[kBatch];
    auto columns = [&](auto* list) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + u * kWarp;
        const int64_t i = k < a.k ? static_cast<int64_t>(list[k]) : -1;
        col[u] = i >= 0 && i < a.cols ? static_cast<int>(i) : -1;
      }
    };
    auto values = [&](auto type, auto* list) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + u * kWarp;
        v[u] = k < a.k ? Score<decltype(type)::value>::load(list[k]) : -INFINITY;
      }
    };
    const int64_t at_i = row * a.index_stride, at_v = row * a.top_stride;
    if (a.top_type == RS_SCORE_BF16)
      values(ScoreTag<RS_SCORE_BF16>{}, static_cast<const uint16_t*>(a.top_values) + at_v);
    else if (a.top_type == RS_SCORE_F16)
      values(ScoreTag<RS_SCORE_F16>{}, static_cast<const uint16_t*>(a.top_values) + at_v);
    else
      values(ScoreTag<RS_SCORE_F32>{}, static_cast<const uint32_t*>(a.top_values) + at_v);
    if (a.index_bytes == 8)
      columns(static_cast<const int64_t*>(a.top_indices) + at_i);
    else
      columns(static_cast<const int32_t*>(a.top_indices) + at_i);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) xi[u] = col[u] >= 0 ? S::load(x[col[u]]) : -INFINITY;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = k0 + u * kWarp;
      if (k < a.k) {
        const float vu = col[u] >= 0 ? v[u] : -INFINITY;
        t.col[k] = col[u];
        t.p[k] = vu;
        t.x[k] = xi[u];
        vm = fmaxf(vm, vu);
        xm = fmaxf(xm, xi[u]);
      }
    }
  }
  vm = origin(warp_max(vm));
  xm = origin(warp_max(xm));
  float sum = 0.0f;
  for (int k = lane; k < a.k; k += kWarp) sum += exp2_approx(apart2(t.p[k], vm, scale2));
  sum = warp_sum(sum);
  const float log_sum = logf(sum);
  float acc = 0.0f;
  for (int k = lane; k < a.k; k += kWarp) {
    const float v = 0.5f * t.p[k] - 0.5f * vm;
    const float p = sum == 0.0f ? 0.0f : exp2_approx(v * (2.0f * scale2)) / sum;
    if (MODE != kLossBwd && p != 0.0f)
      acc += p * (2.0f * kPart * v - kPart * a.tau * log_sum - (kPart * t.x[k] - kPart * xm));
    t.p[k] = p;
  }
  if (MODE != kLossBwd) acc = warp_sum(acc);
  // A column named twice: its first entry gets the sum, in the entries'
  // order, and the others are dropped.  Lists of a sort name none twice, so
  // the columns are first matched across the warp, or looked up in a table;
  // only a list that does repeat one is compared entry by entry.
  if (MODE != kLossFwd && a.k > 1) {
    bool twice = false;
    if (a.k <= kWarp) {
      const int col = lane < a.k ? t.col[lane] : -1;
      const unsigned same = __match_any_sync(kFull, col);
      twice = col >= 0 && (same & (same - 1)) != 0;
    } else {
      const int n = target_slots(a.k);
      for (int i = lane; i < n; i += kWarp) slots[i] = -1;
      __syncwarp();
      for (int k = lane; k < a.k; k += kWarp) {
        const int col = t.col[k];
        if (col < 0) continue;
        int at = static_cast<int>((static_cast<uint32_t>(col) * 2654435769u) >> 7) & (n - 1);
        for (int probe = 0; probe < n; ++probe) {  // the table is at most half full
          const int was = atomicCAS(&slots[at], -1, col);
          if (was == -1) break;
          if (was == col) {
            twice = true;
            break;
          }
          at = (at + 1) & (n - 1);
        }
      }
    }
    if (__any_sync(kFull, twice)) {
      __syncwarp();
      for (int k = lane; k < a.k; k += kWarp) {
        const int col = t.col[k];
        float p = 0.0f;
        bool first = true;
        for (int j = 0; j < a.k; ++j) {
          if (t.col[j] == col) {
            if (j < k) first = false;
            p += t.p[j];
          }
        }
        slots[k] = __float_as_int(first ? p : -1.0f);
      }
      __syncwarp();
      for (int k = lane; k < a.k; k += kWarp) {
        const float p = __int_as_float(slots[k]);
        if (p < 0.0f) t.col[k] = -1;
        t.p[k] = p;
      }
    }
  }
  if (lane == 0) {
    h->off = 0;
    h->live = !(sum == 0.0f);
    h->w = w;
    h->up = up;
    h->a = acc;
    h->ref = xm;
  }
}

// Loss, log-probability and coefficient of a row from its statistics.
struct RowResult {
  float loss, logp, lse, c;
};

// kLossBwd: m is the saved lse (none that far_lse() names), sum is 1.
template <int OP, int MODE>
__device__ __forceinline__ RowResult row_result(const RowLossArgs& a, const Head& h, float m,
                                                float sum) {
  RowResult r;
  const bool empty = MODE != kLossBwd && sum == 0.0f;
  const float log_sum = MODE == kLossBwd ? 0.0f : logf(sum);
  r.lse = empty ? -INFINITY : m * a.inv_tau + log_sum;
  if (OP == kOpDistill) {
    const bool none = empty || !h.live;
    r.logp = 0.0f;
    r.loss = none ? 0.0f
                  : a.tau * h.w *
                        (h.a + (kPart * m - kPart * h.ref + kPart * a.tau * log_sum)) / kPart;
    r.c = none ? 0.0f : h.up * a.tau;
  } else {
    const float logp = empty               ? -INFINITY
                       : MODE == kLossBwd ? h.x0 / a.tau - m
                                          : (0.5f * h.x0 - 0.5f * m) * (2.0f * a.inv_tau) - log_sum;
    const float adv = h.adv;
    const float ratio = expf(logp - h.old);
    const bool held = (adv > 0.0f && ratio > a.clip_high) || (adv < 0.0f && ratio < a.clip_low);
    // an advantage of 0 takes no part, however large the ratio
    const float clipped = fminf(fmaxf(ratio, a.clip_low), a.clip_high);
    float loss = adv == 0.0f ? 0.0f : -(held ? clipped : ratio) * adv;
    float g = held || adv == 0.0f ? 0.0f : -adv * ratio;
    if (isnan(ratio)) loss = g = ratio;
    if (a.ref_logprobs != nullptr) {
      const float d = h.ref_logp - logp;
      const float e = expm1f(d);
      loss += a.kl_coef * (e - d);
      g -= a.kl_coef * e;
    }
    r.logp = logp;
    r.loss = empty ? 0.0f : h.w * loss;
    r.c = empty ? 0.0f : -h.up * g * a.inv_tau;
  }
  return r;
}

// The exponentials of a row from its maximum, or (kLossBwd) its saved lse.
template <int TYPE, int MODE>
__device__ __forceinline__ auto exponent(const RowLossArgs& a, float m) {
  if constexpr (MODE == kLossBwd)
    return ExponentOfLse<TYPE == RS_SCORE_F32>(m, a.scale2, a.scale2_low);
  else
    return Exponent(origin(m), a.scale2);
}

template <int OP>
__device__ __forceinline__ void store_result(const RowLossArgs& a, int64_t row,
                                             const RowResult& r) {
  a.losses[row] = r.loss;
  a.lse[row] = r.lse;
  if (OP == kOpPolicy) a.logprobs[row] = r.logp;
}

__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void store_peer(Softmax* at, uint32_t rank, const Softmax& v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer_addr(smem_addr(at), rank)),
               "f"(v.m), "f"(v.sum)
               : "memory");
}

// The two halves of a cluster's barrier, where it only has to be known that
// every CTA has begun: another CTA's shared memory must not be touched before.
__device__ __forceinline__ void cluster_begun() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The backward call's gradient of vectors [begin, end) of a row whose saved lse
// says too little: the first WARPS warps of the CTA take the statistics of all
// of the row, then its threads write the gradient, one vector at a time.
// Rare, and out of the way of the registers of the usual way (inlined, 8,000 x
// 7,000 policy rows of ordinary lse took 38 us instead of 34).  together: other
// CTAs read the row too, and the gradient goes over it.
template <int TYPE, int OP, int WARPS>
__device__ __noinline__ void backward_again(const RowLossArgs& a, int64_t row, int begin, int end,
                                            Targets t, const Head& head, Softmax* part,
                                            bool together) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  using V = ScoreVec<TYPE>;
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  Raw* g = static_cast<Raw*>(a.grad) + row * a.grad_stride;
  const RowVecs<TYPE> vecs(x, static_cast<int>(a.cols));
  const uint4* xv = reinterpret_cast<const uint4*>(x - vecs.lead);
  const RowOut<TYPE> out(g, vecs);
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  if (tid < WARPS * kWarp) {
    constexpr int kBatch = 2, kStep = WARPS * kWarp;  // more would take registers
    RunningSoftmax<TYPE> run(a.scale2);
#pragma unroll 1
    for (int v0 = tid; v0 < vecs.count; v0 += kBatch * kStep) {
      uint4 r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) r[u] = vecs.load(xv, x, v0 + u * kStep);
      run.add(r);
    }
    const Softmax s = warp_join(run.result(), a.scale2);
    if (lane == 0) part[tid / kWarp] = s;
  }
  __syncthreads();
  const Softmax s = warp_join(lane < WARPS ? part[lane] : Softmax{-INFINITY, 0.0f}, a.scale2);
  const RowResult res = row_result<OP, kLossGrad>(a, head, s.m, s.sum);
  if (together) cluster_sync();
  const float f = res.c / s.sum;
  const Exponent e(origin(s.m), a.scale2);
  const uint64_t ff = pack2(f * e.mend, f * e.mend);
#pragma unroll 1
  for (int v = begin + tid; v < end; v += static_cast<int>(blockDim.x))
    out.store(vecs, v, res.c == 0.0f ? make_uint4(0, 0, 0, 0)
                                     : vec_grad<TYPE>(vecs.load(xv, x, v), e, ff));
  if (res.c == 0.0f) return;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(begin) * V::kCount - vecs.lead;
  const int64_t last = static_cast<int64_t>(end) * V::kCount - vecs.lead;
  for (int k = tid; k < a.k; k += static_cast<int>(blockDim.x)) {
    const int col = t.col[k];
    if (col >= 0 && col >= first && col < last)
      g[col] = S::store(e.one(t.x[k]) * f - res.c * t.p[k]);
  }
}

// ---------------------------------------------------------------- short rows
// One CTA per row, the row in registers: rows of at most kThreads * VECS
// 16-byte vectors.  Many CTAs per SM hide each other's loads and reductions:
// as few threads per row as 8 vectors each allow, and registers held to what
// 24 warps per SM leave (bf16 policy gradients of 8,000 x 7,000 took 50 us; 56
// with 20 warps, 52 with 32, and 78 by 256 threads per row; 16,384 x 16,000
// 191 us, 236 with 20 warps; one after another they take 45 and 178).  What
// bounds it is the chain of a CTA (targets, maximum, sum, gradient) against
// the few KB it moves: 33 and 154 us are the times of the bytes.
constexpr int kShortWarps = 24;
template <int TYPE, int OP, int MODE, int kThreads, int VECS>
__global__ void __launch_bounds__(kThreads, VECS == 16 ? 2 : kShortWarps / (kThreads / kWarp))
    row_loss_short_kernel(const __grid_constant__ RowLossArgs a) {
  grid_dependency_sync();
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  using V = ScoreVec<TYPE>;
  constexpr int kWarps = kThreads / kWarp;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Softmax part[kWarps];
  __shared__ Head head;
  Targets t;
  t.col = reinterpret_cast<int*>(smem);
  t.p = reinterpret_cast<float*>(t.col + a.k);
  t.x = t.p + a.k;
  int* slots = reinterpret_cast<int*>(t.x + a.k);
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int64_t row = blockIdx.x;
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  Raw* g = static_cast<Raw*>(a.grad) + row * a.grad_stride;
  const RowVecs<TYPE> vecs(x, static_cast<int>(a.cols));
  const uint4* xv = reinterpret_cast<const uint4*>(x - vecs.lead);
  const RowOut<TYPE> out(g, vecs);
  const float scale2 = a.scale2;
  if (row_off<OP>(a, row)) {
    if (MODE != kLossBwd && tid == 0) store_result<OP>(a, row, RowResult{0, 0, 0, 0});
    if (MODE != kLossFwd)
      for (int v = tid; v < vecs.count; v += kThreads) out.store(vecs, v, make_uint4(0, 0, 0, 0));
    return;
  }
  uint4 r[VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) r[u] = vecs.load(xv, x, tid + u * kThreads);
  if (warp == kWarps - 1) load_targets<TYPE, OP, MODE>(a, row, t, slots, &head);
  Softmax s;
  if constexpr (MODE == kLossBwd) {
    s = {a.lse[row], 1.0f};
    __syncthreads();
    if (far_lse(s.m))
      return backward_again<TYPE, OP, kWarps>(a, row, 0, vecs.count, t, head, part, false);
  } else {
    s = warp_join(softmax_of<TYPE>(r, scale2), scale2);
    if (lane_id() == 0) part[warp] = s;
    __syncthreads();
    s = lane_id() < kWarps ? part[lane_id()] : Softmax{-INFINITY, 0.0f};
    s = warp_join(s, scale2);
  }
  const RowResult res = row_result<OP, MODE>(a, head, s.m, s.sum);
  if (MODE != kLossBwd && tid == 0) store_result<OP>(a, row, res);
  if (MODE == kLossFwd) return;
  const float f = res.c / s.sum;
  const auto e = exponent<TYPE, MODE>(a, s.m);
  const uint64_t ff = pack2(f * e.mend, f * e.mend);
#pragma unroll
  for (int u = 0; u < VECS; ++u) {
    const int v = tid + u * kThreads;
    if (v < vecs.count)
      out.store(vecs, v, res.c == 0.0f ? make_uint4(0, 0, 0, 0) : vec_grad<TYPE>(r[u], e, ff));
  }
  if (res.c == 0.0f) return;
  __syncthreads();
  for (int k = tid; k < a.k; k += kThreads)
    if (t.col[k] >= 0)
      g[t.col[k]] = S::store(e.one(t.x[k]) * f - res.c * t.p[k]);
}

// -------------------------------------------- long rows, one pass over a row
// The losses alone, and the backward call, read a row once and keep nothing
// of it: plain wide loads, a batch of them always ahead of the arithmetic,
// with three CTAs per SM (batches of 4 vectors; 3 with four CTAs took 101 us
// instead of 83 for a bf16 forward of 2,048 x 131,072, 8 with two 85; the
// ring of the one-call form below 88 to 92).  One more warp reads the row's
// targets meanwhile.  A row is cut into `split` segments of at least 16 KB
// until there are two CTAs for every place on the GPU: four times as many
// CTAs gain nothing (each pays for its targets), sixteen cost 30% and more.
// What bounds them is HBM (69 us for the bytes of that forward), and the last
// CTAs of a grid, which have the GPU to themselves.
constexpr int kStreamThreads = 256;
constexpr int kStreamWarps = kStreamThreads / kWarp;
constexpr int kStreamBatch = 4;   // vectors per thread under way
constexpr int kStreamCtas = 3;    // per SM
constexpr int kStreamWaves = 2;
constexpr int64_t kStreamLeast = 16384;
constexpr int kMaxCluster = 16;

// A thread's vectors of a segment [begin, end): begin + tid, + kStreamThreads,
// ..., in batches of kStreamBatch, the next batch's loads under way while one
// is worked on; vectors past the end are -inf.
template <int TYPE>
struct Stream {
  using Raw = typename Score<TYPE>::Raw;
  using V = ScoreVec<TYPE>;
  static constexpr int kStep = kStreamThreads * kStreamBatch;
  const Raw* x;
  const RowVecs<TYPE>& vecs;
  const int end;
  int v;
  uint4 r[kStreamBatch];

  __device__ __forceinline__ Stream(const Raw* x_, const RowVecs<TYPE>& vecs_, int begin, int end_,
                                    int tid)
      : x(x_), vecs(vecs_), end(end_), v(begin + tid) {
    if (v < end) load(v, r);
  }
  __device__ __forceinline__ void load(int v0, uint4 (&to)[kStreamBatch]) const {
    const uint4* xv = reinterpret_cast<const uint4*>(x - vecs.lead);
    const int v1 = v0 + (kStreamBatch - 1) * kStreamThreads;
    if (v0 >= vecs.whole_begin() && v1 < min(end, vecs.whole_end())) {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) to[u] = __ldcs(xv + v0 + u * kStreamThreads);
    } else {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) {
        const int w = v0 + u * kStreamThreads;
        if (w >= end)
          to[u] = make_uint4(V::kMinusInf, V::kMinusInf, V::kMinusInf, V::kMinusInf);
        else if (vecs.whole(w))
          to[u] = __ldcs(xv + w);
        else
          to[u] = vecs.load_edge(x, w);
      }
    }
  }
  // body(v, vectors) for every batch
  template <class F>
  __device__ __forceinline__ void run(F&& body) {
    uint4 ahead[kStreamBatch];
    for (; v < end; v += kStep) {
      if (v + kStep < end) load(v + kStep, ahead);
      body(v, r);
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) r[u] = ahead[u];
    }
  }
};

template <int TYPE, int OP>
__global__ void __launch_bounds__(kStreamThreads + kWarp, kStreamCtas)
    row_loss_forward_kernel(const RowLossArgs a, const int split) {
  using Raw = typename Score<TYPE>::Raw;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Softmax part[kStreamWarps], peer[kMaxCluster];
  __shared__ Head head;
  grid_dependency_sync();
  Targets t;
  t.col = reinterpret_cast<int*>(smem);
  t.p = reinterpret_cast<float*>(t.col + a.k);
  t.x = t.p + a.k;
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int lane = static_cast<int>(lane_id());
  const int64_t row = blockIdx.x / split;
  const int rank = static_cast<int>(blockIdx.x % split);
  if (row_off<OP>(a, row)) {  // the whole cluster's answer
    if (rank == 0 && tid == 0) store_result<OP>(a, row, RowResult{0, 0, 0, 0});
    return;
  }
  if (split > 1) cluster_begun();
  const float scale2 = a.scale2;
  if (warp == kStreamWarps) {
    if (rank == 0) load_targets<TYPE, OP, kLossFwd>(a, row, t, nullptr, &head);
  } else {
    const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
    const RowVecs<TYPE> vecs(x, static_cast<int>(a.cols));
    const int per = (vecs.count + split - 1) / split;
    const int begin = min(rank * per, vecs.count), end = min(begin + per, vecs.count);
    RunningSoftmax<TYPE> run(scale2);
    Stream<TYPE> stream(x, vecs, begin, end, tid);
    stream.run([&](int, const uint4(&r)[kStreamBatch]) { run.add(r); });
    const Softmax s = warp_join(run.result(), scale2);
    if (lane == 0) part[warp] = s;
  }
  __syncthreads();
  Softmax s{-INFINITY, 0.0f};
  if (warp == 0) s = warp_join(lane < kStreamWarps ? part[lane] : s, scale2);
  if (split > 1) {
    cluster_wait();
    if (tid == 0) store_peer(&peer[rank], 0, s);
    cluster_sync();
    if (rank != 0) return;
    if (warp == 0) s = warp_join(lane < split ? peer[lane] : Softmax{-INFINITY, 0.0f}, scale2);
  }
  if (tid == 0) store_result<OP>(a, row, row_result<OP, kLossFwd>(a, head, s.m, s.sum));
}

template <int TYPE, int OP>
__global__ void __launch_bounds__(kStreamThreads + kWarp, kStreamCtas)
    row_loss_backward_kernel(const __grid_constant__ RowLossArgs a, const int split,
                             const bool together) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  using V = ScoreVec<TYPE>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Softmax part[kStreamWarps];
  __shared__ Head head;
  grid_dependency_sync();
  Targets t;
  t.col = reinterpret_cast<int*>(smem);
  t.p = reinterpret_cast<float*>(t.col + a.k);
  t.x = t.p + a.k;
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int64_t row = blockIdx.x / split;
  const int rank = static_cast<int>(blockIdx.x % split);
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  Raw* g = static_cast<Raw*>(a.grad) + row * a.grad_stride;
  const RowVecs<TYPE> vecs(x, static_cast<int>(a.cols));
  const int per = (vecs.count + split - 1) / split;
  const int begin = min(rank * per, vecs.count), end = min(begin + per, vecs.count);
  const RowOut<TYPE> out(g, vecs);
  const int inner_end = min(end, vecs.whole_end());
  auto put = [&](int v0, const uint4(&r)[kStreamBatch]) {
    // the same for all lanes of the warp
    const int first = v0 - static_cast<int>(lane_id());
    const bool inner = first >= vecs.whole_begin() &&
                       first + (kStreamBatch - 1) * kStreamThreads + kWarp <= inner_end;
    if (inner && out.shift == 0) {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) __stcs(out.vec0 + v0 + u * kStreamThreads, r[u]);
    } else if (inner) {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) out.store_shifted(v0 + u * kStreamThreads, r[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) {
        const int v = v0 + u * kStreamThreads;
        if (v < end) out.store(vecs, v, r[u]);
      }
    }
  };
  const bool off = row_off<OP>(a, row);
  if (warp == kStreamWarps && !off)
    load_targets<TYPE, OP, kLossBwd>(a, row, t, reinterpret_cast<int*>(t.x + a.k), &head);
  // the first loads are under way before the targets are known
  Stream<TYPE> stream(x, vecs, begin, off || warp == kStreamWarps ? begin : end, tid);
  const float m = off ? 0.0f : a.lse[row];
  __syncthreads();
  if (far_lse(m))
    return backward_again<TYPE, OP, kStreamWarps>(a, row, begin, end, t, head, part, together);
  const float c = off ? 0.0f : row_result<OP, kLossBwd>(a, head, m, 1.0f).c;
  const auto e = exponent<TYPE, kLossBwd>(a, m);
  // over its own logits no CTA of the row may write before all of them have
  // read the action's score
  if (together && !off) cluster_sync();
  if (warp < kStreamWarps) {
    if (c == 0.0f) {  // nothing of the row is read
      const uint4 zero[kStreamBatch] = {};
      for (int v = begin + tid; v < end; v += kStreamThreads * kStreamBatch) put(v, zero);
    } else {
      const uint64_t f = pack2(c * e.mend, c * e.mend);
      stream.run([&](int v, uint4(&r)[kStreamBatch]) {
#pragma unroll
        for (int u = 0; u < kStreamBatch; ++u) r[u] = vec_grad<TYPE>(r[u], e, f);
        put(v, r);
      });
    }
  }
  if (c == 0.0f) return;
  __syncthreads();  // the targets' columns are written last
  const int64_t b = static_cast<int64_t>(begin) * V::kCount - vecs.lead;
  const int64_t last = static_cast<int64_t>(end) * V::kCount - vecs.lead;
  for (int k = tid; k < a.k; k += kStreamThreads + kWarp) {
    const int col = t.col[k];
    if (col >= 0 && col >= b && col < last)
      g[col] = S::store(e.one(t.x[k]) * c - c * t.p[k]);
  }
}

// ------------------------------------- long rows, losses and gradient at once
// One CTA holds a row: a producer warp copies it by TMA bulk copies, in chunks
// of 32 KB, into a ring of shared-memory slots, row after row, as far ahead as
// slots are free; two warps read the next rows' targets; 16 warps go over the
// row's chunks twice: once for the maximum and the sum, and once more to write
// the gradient, freeing the slots for the next row.  All but one of the ring's
// slots may hold chunks of the row between the two passes (160 KB; the other
// is what the copies go on through); what does not fit is copied again, from
// L2.  So memory is read once, and the copies never stop for the arithmetic.
//
// Rows of more than twice the ring, and rows too few for the SMs, are shared
// by the `split` CTAs of a cluster, which exchange maxima and sums through
// distributed shared memory.  That exchange costs more than the second copy
// from L2: bf16 rows of 131,072 took 443 us for 4,096 rows as clusters of two
// that keep everything, 326 us as single CTAs that copy 96 of 256 KB again.
// Chunks of 16 KB, every wait and release twice as often, took 361 us for
// 8,192 rows of 65,536 instead of 339; per-warp rings of 2 KB copies 437,
// per-thread cp.async rings 434 (each pair measured in one run).
//
// What bounds it is HBM: 329 us for the distillation loss and gradient of
// 4,096 x 131,072 with an eighth of the rows masked (90% of the measured copy
// bandwidth), 320 us for the policy loss of 8,192 x 65,536 (93%).  Rows of
// little more than a chunk or two pay for the exchange between their passes
// (3,000 x 49,152: 107 us, 81%).
//
// Rows cost unequally (a masked row is not read), so they are not dealt out
// beforehand: the grid has a CTA (cluster) per row, and a running one takes
// over the rows of CTAs that have not been launched yet, one row after
// another, by cancelling their launch (cluster launch control).  One thread
// per CTA (the scheduler; the first CTA's asks and tells the others') does so
// a few rows ahead and lists them for the other warps.
//
// Every wait has a limit.  One that runs out marks the whole cluster as
// failed; its warps then finish the row they are in, on whatever data, and
// leave.  Copies and answers under way are waited for; nothing is in flight
// when a CTA ends.  The rows taken over are no other CTA's any more, so those
// that some warp has not finished in good order get NaN, all of them, and the
// caller's status word is set.
constexpr int kRowConsumers = 512;
constexpr int kRowWarps = kRowConsumers / kWarp;
constexpr int kTargetWarps = 2;
constexpr int kProducerWarp = kRowWarps, kSchedulerWarp = kRowWarps + 1,
              kFirstTargetWarp = kRowWarps + 2;
constexpr int kRowThreads = kRowConsumers + (2 + kTargetWarps) * kWarp;
constexpr int kChunkUnits = 4;                                // vectors per thread and chunk
constexpr int kChunkVecs = kRowConsumers * kChunkUnits;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kMaxSlots = 6;                                  // most ring slots
constexpr int kMaxHeads = 4;                                  // rows whose targets are held
// Rows that the scheduler is ahead: enough for the targets, and not more, or
// the last rows pile up at few CTAs (8: bf16 4,096 x 131,072 with 64 targets
// 337 us instead of 330, 300 x 400,000 106 instead of 98).
constexpr int kAheadRows = 4;
constexpr int kRowReaders = kRowWarps + 1 + kTargetWarps;     // warps that read its list
// Rows that are remembered.  A scheduler lists row n once every warp of its CTA
// has begun row n - kAheadRows, and the first CTA's remembers row n for all
// once the others' have read row n - kTold, or n - kTold - 1 where that wait
// gives up: no row before n - kAheadRows - kTold - 2 is unfinished then.
constexpr int kTold = 2;
constexpr int kRowHistory = 16;
static_assert(kRowHistory >= kAheadRows + kTold + 3 && kRowHistory % kAheadRows == 0);

// Barriers and small arrays behind the ring.
struct RowShared {
  uint4 answer;                                               // of cluster launch control
  uint64_t answer_full;
  uint64_t told_full[kTold], told_empty[kTold];
  uint64_t row_full[kAheadRows], row_empty[kAheadRows];
  int2 row[kRowHistory];  // row n at n % kRowHistory: its number (-1: no more), and whether it
                          // is not read
  int taken;              // rows taken so far by the cluster
  int done[kRowWarps];    // rows that a consumer warp has finished
  int first_bad;          // the least of these in the cluster
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t head_full[kMaxHeads], head_empty[kMaxHeads];
  uint64_t together;                                          // all consumer warps
  uint64_t peers;                                             // exchange of the CTAs' softmaxes
  Softmax part[2][kRowWarps];
  Softmax peer[2][kMaxCluster];
  Head head[kMaxHeads];
  int failed;                                                 // a wait of the cluster ran out
};

// Rows whose targets are held at a time (with two, 64 targets a row took 387
// us for 8,192 rows of 65,536 instead of 337; long lists leave no room for
// four), their lists, and a table per target warp.
__host__ __device__ constexpr inline int row_heads(int k) { return k <= 256 ? kMaxHeads : 2; }
__host__ __device__ constexpr inline size_t row_list_bytes(int k) {
  return align_up(static_cast<size_t>(k) * 12, 16);
}
__host__ constexpr inline size_t row_ring_smem(int k, int slots) {
  return static_cast<size_t>(slots) * kChunkBytes + align_up(sizeof(RowShared), 16) +
         row_heads(k) * row_list_bytes(k) + static_cast<size_t>(kTargetWarps) * target_slots(k) * 4;
}
// As many slots as fit beside the lists of k entries.
constexpr size_t kMaxSmem = 232448;
__host__ constexpr inline int row_ring_slots(int k) {
  int n = kMaxSlots;
  while (row_ring_smem(k, n) > kMaxSmem) --n;
  return n;
}

// Waits for a phase of a barrier, with CLUSTER for one on which other CTAs
// arrive (what they wrote before is then seen after it).  It gives up after
// limit_ns, or once another wait has.  Each try names a time to sleep: warps
// that poll in a tight loop take the issue slots and the shared-memory ports
// of those that work (a 4096 x 131072 bf16 gradient took 500 us so, 441 with a
// read of the clock between polls).
template <bool CLUSTER>
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity, uint32_t sleep_ns) {
  uint32_t ok;
  if (CLUSTER)
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(sleep_ns)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(sleep_ns)
        : "memory");
  return ok != 0;
}
enum WaitResult { kWaitDone, kWaitFailedBefore, kWaitRanOut };
template <bool CLUSTER>
__device__ __forceinline__ WaitResult wait_phase(uint64_t* bar, uint32_t parity,
                                                 const volatile int* failed, uint64_t limit_ns,
                                                 uint32_t sleep_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!phase_done<CLUSTER>(bar, parity, sleep_ns)) {
    if (*failed) return kWaitFailedBefore;
    if (global_timer_ns() - t0 > limit_ns) return kWaitRanOut;
  }
  return kWaitDone;
}

__device__ __forceinline__ void store_peer(int* at, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(peer_addr(smem_addr(at), rank)), "r"(v)
               : "memory");
}
__device__ __forceinline__ void store_peer(int2* at, uint32_t rank, int2 v) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(peer_addr(smem_addr(at), rank)),
               "r"(v.x), "r"(v.y)
               : "memory");
}
__device__ __forceinline__ int load_peer(const int* at, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];"
               : "=r"(v)
               : "r"(peer_addr(smem_addr(at), rank))
               : "memory");
  return v;
}

// The rest of a wait whose first try did not end in time, out of the way of
// the code around it (inlined everywhere it cost the policy case 2%).
template <bool CLUSTER>
__device__ __noinline__ bool wait_longer(RowShared* sh, uint64_t* bar, uint32_t parity,
                                         uint64_t limit_ns, uint32_t sleep_ns, int split) {
  const WaitResult w = wait_phase<CLUSTER>(bar, parity, &sh->failed, limit_ns, sleep_ns);
  if (w == kWaitRanOut)  // for the whole cluster
    for (int r = 0; r < split; ++r) store_peer(&sh->failed, r, 1);
  return w == kWaitDone;
}

// One thread's waits in the ring kernel.
struct RowWaits {
  RowShared* sh;
  uint64_t limit_ns;
  uint32_t sleep_ns;
  int split;

  __device__ __forceinline__ RowWaits(RowShared* sh_, uint64_t limit, int split_)
      : sh(sh_),
        limit_ns(limit),
        sleep_ns(limit < 1000000 ? static_cast<uint32_t>(limit) : 1000000u),
        split(split_) {}
  template <bool CLUSTER>
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return phase_done<CLUSTER>(bar, parity, sleep_ns) ||
           wait_longer<CLUSTER>(sh, bar, parity, limit_ns, sleep_ns, split);
  }
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    return wait<false>(bar, parity);
  }
  // all lanes of a warp, which agree on the outcome
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(kFull, wait<false>(bar, parity));
  }
  __device__ __forceinline__ bool warp_cluster(uint64_t* bar, uint32_t parity) const {
    return __all_sync(kFull, wait<true>(bar, parity));
  }
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Arrives on a barrier of any CTA of the cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}

// Asks for the launch of a CTA (cluster) that has not begun yet to be
// cancelled; the answer (16 bytes) arrives in this CTA's shared memory.
__device__ __forceinline__ void ask_next(uint4* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(smem_addr(answer)),
      "r"(smem_addr(bar))
      : "memory");
}

// The first CTA of the cancelled launch, or -1: nothing was left.
__device__ __forceinline__ int next_cta(const uint4* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n .reg .b32 y, z, w;\n"
      " ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n"
      " mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  // the answer has been read before the next one may be written there
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return ok != 0 ? static_cast<int>(x) : -1;
}

template <int TYPE, int OP>
__global__ void __launch_bounds__(kRowThreads, 1)
    row_loss_ring_kernel(const RowLossArgs a, const int split, const int ring_slots,
                         const bool steal) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  using V = ScoreVec<TYPE>;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* ring = smem;
  RowShared* sh = reinterpret_cast<RowShared*>(smem + ring_slots * kChunkBytes);
  unsigned char* lists = reinterpret_cast<unsigned char*>(sh) + align_up(sizeof(RowShared), 16);
  auto targets = [&](int i) {
    Targets t;
    t.col = reinterpret_cast<int*>(lists + i * row_list_bytes(a.k));
    t.p = reinterpret_cast<float*>(t.col + a.k);
    t.x = t.p + a.k;
    return t;
  };
  const int heads = row_heads(a.k);
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(blockIdx.x) % split;  // in the cluster
  const RowWaits wait(sh, a.wait_ns, split);
  // vectors per CTA, whatever the row's first address
  const int per = (static_cast<int>(a.cols + 2 * (V::kCount - 1)) / V::kCount + split - 1) / split;
  if (tid == 0) {
    for (int i = 0; i < ring_slots; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], kRowWarps);
    }
    for (int i = 0; i < heads; ++i) {
      mbar_init(&sh->head_full[i], 1);
      mbar_init(&sh->head_empty[i], kRowWarps);
    }
    mbar_init(&sh->answer_full, 1);
    for (int i = 0; i < kAheadRows; ++i) {
      mbar_init(&sh->row_full[i], 1);
      mbar_init(&sh->row_empty[i], kRowReaders);
    }
    for (int i = 0; i < kTold; ++i) {
      mbar_init(&sh->told_full[i], 1);
      mbar_init(&sh->told_empty[i], split > 1 ? split - 1 : 1);
    }
    mbar_init(&sh->together, kRowWarps);
    mbar_init(&sh->peers, split);
    sh->failed = 0;
    sh->row[0] = make_int2(static_cast<int>(blockIdx.x) / split, 0);
    sh->taken = 1;  // the row that the CTA was launched for
    sh->first_bad = INT_MAX;
  }
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  grid_dependency_sync();

  // One warp's way through the scheduler's list: the next row, or -1.
  struct Way {
    uint32_t n;  // rows so far
    bool off;    // the row is not read
  };
  auto next_row = [&](Way& way) {
    const uint32_t at = way.n % kAheadRows, phase = way.n / kAheadRows & 1;
    if (!wait.warp(&sh->row_full[at], phase)) return -1;
    const int2 row = sh->row[way.n++ % kRowHistory];
    way.off = row.y != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->row_empty[at]);
    return row.x;
  };
  // This CTA's segment of a row: vectors [begin, end), in chunks, the last
  // `keep` of which stay in the ring for the second pass.
  struct Segment {
    const Raw* x;
    RowVecs<TYPE> vecs;
    int begin, end, chunks, keep;
  };
  auto segment = [&](int64_t row) {
    const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
    Segment s{x, RowVecs<TYPE>(x, static_cast<int>(a.cols)), 0, 0, 0, 0};
    s.begin = min(rank * per, s.vecs.count);
    s.end = min(s.begin + per, s.vecs.count);
    s.chunks = (s.end - s.begin + kChunkVecs - 1) / kChunkVecs;
    s.keep = min(s.chunks, ring_slots - 1);
    return s;
  };

  if (warp == kProducerWarp) {
    int slot = 0;
    uint32_t use = 0;        // times round the ring
    uint32_t put_by_us = 0;  // slots (bits) that hold scores stored by this warp
    Way way{0, false};
    bool going = true;
    for (int row; going && (row = next_row(way)) >= 0;) {
      if (way.off) continue;
      const Segment s = segment(row);
      const uint4* xv = reinterpret_cast<const uint4*>(s.x - s.vecs.lead);
      const int tail = s.vecs.count - 1;  // the last vector, and whether it is part of the row
      const bool ragged_tail = s.vecs.whole_end() < s.vecs.count;
      // every chunk, then those that do not stay once more
      for (int i = 0; i < 2 * s.chunks - s.keep; ++i) {
        const int first = s.begin + (i < s.chunks ? i : i - s.chunks) * kChunkVecs;
        const int last = min(first + kChunkVecs, s.end);
        const int b = max(first, s.vecs.whole_begin()), e = min(last, s.vecs.whole_end());
        unsigned char* to = ring + slot * kChunkBytes;
        bool ok = true;
        if (lane == 0) {
          if (use > 0) ok = wait(&sh->empty[slot], (use - 1) & 1);
          if (ok && e > b) {
            // plain stores to a slot come before the bulk copy over it, which
            // is of another proxy
            if (put_by_us >> slot & 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_expect_tx(&sh->full[slot], static_cast<uint32_t>(e - b) * 16u);
            bulk_copy_g2s(to + (b - first) * 16, xv + b, static_cast<uint32_t>(e - b) * 16u,
                          &sh->full[slot]);
          }
        }
        going = __shfl_sync(kFull, ok, 0);
        if (!going) break;
        // Vectors at the row's ends that are not whole are put together here,
        // one lane per score, ahead of the warps that would wait for each load
        // (3,000 bf16 rows of 49,153 took 153 us so, 49,152 took 116).
        if (e > b) put_by_us &= ~(1u << slot);
        if (s.vecs.lead != 0 && first == 0) {
          s.vecs.copy_edge(s.x, 0, to, lane);
          put_by_us |= 1u << slot;
        }
        if (ragged_tail && tail >= first && tail < last && (tail != 0 || s.vecs.lead == 0)) {
          s.vecs.copy_edge(s.x, tail, to + (tail - first) * 16, lane);
          put_by_us |= 1u << slot;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->full[slot]);
        if (++slot == ring_slots) {
          slot = 0;
          ++use;
        }
      }
    }
    if (lane == 0)  // copies in flight end before the CTA does, whoever else has left
      for (int i = 0; i < ring_slots; ++i)
        if (i < slot || use > 0)
          mbar_wait_bounded(&sh->full[i], (i < slot ? use : use - 1) & 1, kCopyDrainNs);
  } else if (warp == kSchedulerWarp) {
    if (lane == 0) {
      int2 row = make_int2(sh->row[0].x, 0);
      row.y = row_off<OP>(a, row.x);
      sh->row[0].y = row.y;
      for (uint32_t n = 0;; ++n) {
        const uint32_t m = n - 1, told = m % kTold;  // from the second row on
        if (n > 0 && rank > 0 && steal) {  // what the first CTA has remembered here
          if (!wait.wait<true>(&sh->told_full[told], m / kTold & 1)) break;
          row = sh->row[n % kRowHistory];
          mbar_arrive_cluster(peer_addr(smem_addr(&sh->told_empty[told]), 0));
        } else if (n > 0 && !steal) {
          sh->row[n % kRowHistory] = row;
        } else if (n > 0) {
          // remembered whatever has happened: no other CTA has the row any more
          const bool ok = m < kTold || split == 1 ||
                          wait.wait<true>(&sh->told_empty[told], (m / kTold - 1) & 1);
          for (int r = split - 1; r >= 0; --r) {
            store_peer(&sh->row[n % kRowHistory], r, row);
            if (row.x >= 0) store_peer(&sh->taken, r, static_cast<int>(n) + 1);
            if (ok && r > 0) mbar_arrive_cluster(peer_addr(smem_addr(&sh->told_full[told]), r));
          }
          if (!ok) break;
        }
        const int at = n % kAheadRows;
        if (n >= kAheadRows && !wait(&sh->row_empty[at], (n / kAheadRows - 1) & 1)) break;
        mbar_arrive(&sh->row_full[at]);
        if (row.x < 0) break;
        row = make_int2(-1, 0);
        if (!steal || rank > 0 || *static_cast<volatile int*>(&sh->failed)) continue;
        mbar_arrive_expect_tx(&sh->answer_full, 16);
        ask_next(&sh->answer, &sh->answer_full);
        if (!mbar_wait_bounded(&sh->answer_full, n & 1, kCopyDrainNs)) {
          for (int r = 0; r < split; ++r) store_peer(&sh->failed, r, 1);
          break;
        }
        const int cta = next_cta(&sh->answer);
        if (cta >= 0) {
          row.x = cta / split;
          row.y = row_off<OP>(a, row.x);
        }
      }
    }
  } else if (warp >= kFirstTargetWarp) {  // every kTargetWarps-th row each
    int* table = reinterpret_cast<int*>(lists + heads * row_list_bytes(a.k)) +
                 (warp - kFirstTargetWarp) * target_slots(a.k);
    Way way{0, false};
    uint32_t n = 0;  // the row's number among those of this CTA that are read
    for (int row; (row = next_row(way)) >= 0;) {
      if (way.off) continue;
      const uint32_t i = n % heads, use = n / heads;
      if (static_cast<int>(n++ % kTargetWarps) != warp - kFirstTargetWarp) continue;
      if (use > 0 && !wait.warp(&sh->head_empty[i], (use - 1) & 1)) break;
      load_targets<TYPE, OP, kLossGrad>(a, row, targets(i), table, &sh->head[i]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->head_full[i]);
    }
  } else {  // ---- consumers
    const float scale2 = a.scale2;
    int slot = 0, hi = 0;
    uint32_t phase = 0, head_phase = 0, parity = 0;  // parity: of the rows read
    // A chunk's vectors of this thread from their slot: all of them, or one
    // (-inf past the segment's end).
    auto fetch = [&](int at, uint4 (&r)[kChunkUnits]) {
      const uint4* from = reinterpret_cast<const uint4*>(ring + at * kChunkBytes) + tid;
#pragma unroll
      for (int u = 0; u < kChunkUnits; ++u) r[u] = from[u * kRowConsumers];
    };
    auto fetch_one = [&](const Segment& s, int at, int u, int v) {
      if (v >= s.end) return make_uint4(V::kMinusInf, V::kMinusInf, V::kMinusInf, V::kMinusInf);
      return reinterpret_cast<const uint4*>(ring + at * kChunkBytes)[tid + u * kRowConsumers];
    };
    // Gives a slot back once every lane holds what it read from it.  Arriving
    // on the barrier does not wait for reads that are still queued (behind
    // stores that memory holds up, for microseconds), and the next copy would
    // overtake them; so which lane arrives depends on the data themselves:
    // `read` joins the ends of every vector read.
    auto release = [&](int at, uint32_t read) {
      const int who = __any_sync(kFull, read == 0x7FADC0DEu) ? 1 : 0;  // either will do
      __syncwarp();
      if (lane == who) mbar_arrive(&sh->empty[at]);
    };
    auto join = [](const uint4 (&r)[kChunkUnits]) {
      uint32_t w = r[0].x ^ r[0].w;
#pragma unroll
      for (int u = 1; u < kChunkUnits; ++u) w ^= r[u].x ^ r[u].w;
      return w;
    };
    Way way{0, false};
    int done = 0;
    for (int row; (row = next_row(way)) >= 0; ++done) {
      const Segment s = segment(row);
      Raw* g = static_cast<Raw*>(a.grad) + row * a.grad_stride;
      const RowOut<TYPE> out(g, s.vecs);
      if (way.off) {
        if (rank == 0 && tid == 0) store_result<OP>(a, row, RowResult{0, 0, 0, 0});
        for (int v = s.begin + tid; v < s.end; v += kRowConsumers)
          out.store(s.vecs, v, make_uint4(0, 0, 0, 0));
        continue;
      }
      const int full_chunks = (s.end - s.begin) / kChunkVecs;
      // of which chunks [inner0, inner1) consist of whole vectors
      const int inner0 = s.begin < s.vecs.whole_begin();
      const int inner1 = max(inner0, (min(s.end, s.vecs.whole_end()) - s.begin) / kChunkVecs);
      const int early = s.chunks - s.keep;  // chunks that do not stay
      const int slot0 = slot;
      const uint32_t phase0 = phase;
      // ---- the maximum and the sum
      RunningSoftmax<TYPE> run(scale2);
      bool lost = false;  // a wait of this thread has run out
      for (int c = 0; c < s.chunks; ++c) {
        lost |= !wait(&sh->full[slot], phase);
        if (c < full_chunks) {
          uint4 r[kChunkUnits];
          fetch(slot, r);
          if (c < early) release(slot, join(r));
          run.add(r);
        } else {
          const int v = s.begin + c * kChunkVecs + tid;
          uint32_t read = 0;
#pragma unroll 1
          for (int u = 0; u < kChunkUnits && v - lane + u * kRowConsumers < s.end; ++u) {
            const uint4 r[1] = {fetch_one(s, slot, u, v + u * kRowConsumers)};
            run.add(r);
            read ^= r[0].x ^ r[0].w;
          }
          if (c < early) release(slot, read);
        }
        if (++slot == ring_slots) {
          slot = 0;
          phase ^= 1;
        }
      }
      // NaN tells every warp of the row to look whether a wait has run out
      Softmax st = warp_join(lost ? Softmax{-INFINITY, NAN} : run.result(), scale2);
      Softmax* part = sh->part[parity];
      if (lane == 0) {
        part[warp] = st;
        mbar_arrive(&sh->together);
      }
      // every consumer warp has come here (a bounded wait, unlike bar.sync)
      bool bad = !wait.warp(&sh->together, parity);
      st = warp_join(lane < kRowWarps ? part[lane] : Softmax{-INFINITY, 0.0f}, scale2);
      // This CTA has read its targets before any CTA of the cluster learns the
      // row's sum: the gradient may lie over the logits, and a CTA's targets
      // are scores of all the others' segments.  (They are read rows ahead:
      // the wait is over as a rule.)
      const bool got_head = wait.warp(&sh->head_full[hi], head_phase);
      if (split > 1) {
        if (tid < split) {  // thread i hands this CTA's part to CTA i
          store_peer(&sh->peer[parity][rank], tid, st);
          mbar_arrive_cluster(peer_addr(smem_addr(&sh->peers), tid));
        }
        bad |= !wait.warp_cluster(&sh->peers, parity);
        st = warp_join(lane < split ? sh->peer[parity][lane] : Softmax{-INFINITY, 0.0f}, scale2);
      }
      parity ^= 1;
      // ---- the coefficient
      const Targets t = targets(hi);
      const RowResult res = row_result<OP, kLossGrad>(a, sh->head[hi], st.m, st.sum);
      if (rank == 0 && tid == 0) store_result<OP>(a, row, res);
      // ---- the gradient: the chunks that stayed, then those copied again
      const float f = res.c / st.sum;
      const Exponent e(origin(st.m), scale2);
      const uint64_t ff = pack2(f * e.mend, f * e.mend);
      int at = slot0 + early;
      uint32_t ph = phase0;
      while (at >= ring_slots) {
        at -= ring_slots;
        ph ^= 1;
      }
      for (int i = 0; i < s.chunks; ++i) {
        const int c = i < s.keep ? early + i : i - s.keep;
        const int begin = s.begin + c * kChunkVecs;
        const bool inner = c >= inner0 && c < inner1;
        if (i >= s.keep) lost |= !wait(&sh->full[at], ph);  // the others: see above
        auto result = [&](const uint4& x) {  // zero also where the row holds NaN
          return res.c == 0.0f ? make_uint4(0, 0, 0, 0) : vec_grad<TYPE>(x, e, ff);
        };
        if (inner) {
          uint4 r[kChunkUnits];
          fetch(at, r);
          release(at, join(r));
#pragma unroll
          for (int u = 0; u < kChunkUnits; ++u) r[u] = result(r[u]);
          if (out.shift == 0) {
#pragma unroll
            for (int u = 0; u < kChunkUnits; ++u) out.vec0[begin + tid + u * kRowConsumers] = r[u];
          } else {
#pragma unroll
            for (int u = 0; u < kChunkUnits; ++u)
              out.store_shifted(begin + tid + u * kRowConsumers, r[u]);
          }
        } else {
          const int lo = s.vecs.whole_begin(), up = min(s.end, s.vecs.whole_end());
          uint32_t read = 0;
#pragma unroll 1
          for (int u = 0; u < kChunkUnits; ++u) {
            const int v = begin + tid + u * kRowConsumers, v0 = v - lane;  // v0: of the warp
            if (v0 >= s.end) break;
            const uint4 x = fetch_one(s, at, u, v), y = result(x);
            read ^= x.x ^ x.w;
            if (out.shift != 0 && v0 >= lo && v0 + kWarp <= up)
              out.store_shifted(v, y);
            else if (v < s.end)
              out.store(s.vecs, v, y);
          }
          release(at, read);
        }
        if (++at == ring_slots) {
          at = 0;
          ph ^= 1;
        }
      }
      slot = at;
      phase = ph;
      // ---- the targets' columns, each by the warp that wrote its vector
      __syncwarp();
      if (res.c != 0.0f && got_head) {
        for (int k = lane; k < a.k; k += kWarp) {
          const int col = t.col[k];
          const int v = (col + s.vecs.lead) / V::kCount - s.begin;  // among the CTA's vectors
          if (col >= 0 && v >= 0 && v < s.end - s.begin && v / kWarp % kRowWarps == warp)
            g[col] = S::store(e.one(t.x[k]) * f - res.c * t.p[k]);
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&sh->head_empty[hi]);
      if (++hi == heads) {
        hi = 0;
        head_phase ^= 1;
      }
      bad |= !got_head || isnan(st.sum);
      if (early > 0) bad |= __any_sync(kFull, lost) != 0;
      // where a wait of the row has run out (and not only a score is NaN) the
      // row is not counted, and the warp leaves
      if (bad && __any_sync(kFull, *static_cast<volatile int*>(&sh->failed))) break;
    }
    if (lane == 0) sh->done[warp] = done;
  }
  // No CTA ends while another may still write into its shared memory; from
  // here on everyone knows whether a wait has run out.
  __syncwarp();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (!sh->failed) return;
  for (int i = tid; i < split * kRowWarps; i += kRowThreads)
    atomicMin(&sh->first_bad, load_peer(&sh->done[i % kRowWarps], i / kRowWarps));
  __syncthreads();
  for (int n = sh->first_bad; n < sh->taken; ++n) {
    const int row = sh->row[n % kRowHistory].x;
    const Segment s = segment(row);
    const RowOut<TYPE> out(static_cast<Raw*>(a.grad) + row * a.grad_stride, s.vecs);
    uint64_t nan[V::kCount / 2];
#pragma unroll
    for (int i = 0; i < V::kCount / 2; ++i) nan[i] = pack2(NAN, NAN);
    for (int v = s.begin + tid; v < s.end; v += kRowThreads)
      out.store(s.vecs, v, vec_of<TYPE>(nan));
    if (rank == 0 && tid == 0) store_result<OP>(a, row, RowResult{NAN, NAN, NAN, NAN});
  }
  if (a.status != nullptr && rank == 0 && tid == 0) *a.status = kErrLookback;
  if (split > 1) cluster_sync();  // nor while another reads it
}

// -------------------------------------------------------------------- launch
// Opts a kernel into what its launches need (all of the shared memory, or
// clusters of 16), once per device.
template <class K>
cudaError_t allow(K kern, bool smem, bool big_cluster, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  if (smem)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMaxSmem));
  if (e == cudaSuccess && big_cluster)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

inline int add_attributes(cudaLaunchAttribute* attr, int cluster) {
  int n = 0;
#if LSDRS_PDL
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
#endif
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  return n;
}

template <int TYPE, int OP, int MODE>
cudaError_t launch_stream(const RowLossArgs& a, int split, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * split));
  cfg.blockDim = dim3(kStreamThreads + kWarp);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  // the CTAs of a row wait for each other in the forward call, and in the
  // backward one over its own logits
  const bool together = split > 1 && (MODE == kLossFwd || a.grad == a.logits);
  cfg.numAttrs = add_attributes(attr, together ? split : 1);
  static std::atomic<uint64_t> done{0};
  auto go = [&](auto kern, auto... args) {
    if (together && split > 8) {
      const cudaError_t e = allow(kern, false, true, &done);
      if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, a, args...);
  };
  if constexpr (MODE == kLossFwd)
    return go(row_loss_forward_kernel<TYPE, OP>, split);
  else
    return go(row_loss_backward_kernel<TYPE, OP>, split, together);
}

template <int TYPE, int OP>
cudaError_t launch_ring(const RowLossArgs& a, int sms, int64_t bytes, cudaStream_t s) {
  const int slots = row_ring_slots(a.k);
  int split = 1;
  while (split < 8 && bytes > int64_t(split) * 2 * slots * kChunkBytes) split *= 2;
  while (split < kMaxCluster && a.rows * split * 2 <= sms && bytes >= int64_t(split) * 2 * 8192)
    split *= 2;
  while (a.rows * split >= (int64_t(1) << 31)) split /= 2;  // CTA numbers are 31 bits
  auto kern = row_loss_ring_kernel<TYPE, OP>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow(kern, true, true, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * split));
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = row_ring_smem(a.k, slots);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = add_attributes(attr, split);
  return cudaLaunchKernelEx(&cfg, kern, a, split, slots, a.rows * split > sms);
}

template <int TYPE, int OP, int MODE>
cudaError_t launch_row_loss_as(const RowLossArgs& a, cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<TYPE>::Raw);
  const int64_t bytes = a.cols * kEs;
  const size_t lists = static_cast<size_t>(a.k) * 12 + static_cast<size_t>(target_slots(a.k)) * 4;
  // vectors of a row: one more where rows begin inside one
  constexpr int kN = ScoreVec<TYPE>::kCount;
  const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                       (a.rows == 1 || a.stride % kN == 0);
  const int64_t vecs = (a.cols + (aligned ? 1 : 2) * (kN - 1)) / kN;
  const dim3 each(static_cast<unsigned>(a.rows));
  if (vecs <= 64 * 4)
    return launch_kernel(row_loss_short_kernel<TYPE, OP, MODE, 64, 4>, each, dim3(64), lists, s, a);
  if (vecs <= 64 * 8)
    return launch_kernel(row_loss_short_kernel<TYPE, OP, MODE, 64, 8>, each, dim3(64), lists, s, a);
  if (vecs <= 128 * 8)
    return launch_kernel(row_loss_short_kernel<TYPE, OP, MODE, 128, 8>, each, dim3(128), lists, s,
                         a);
  if (vecs <= 256 * 8)
    return launch_kernel(row_loss_short_kernel<TYPE, OP, MODE, 256, 8>, each, dim3(256), lists, s,
                         a);
  const int sms = device_sm_count();
  // Rows of 32 to 64 KB, where they outnumber the SMs (the ring holds one per
  // SM, registers two): f16 policy gradients of 160 x 30,000 took 7.8 us so and
  // 11.6 in the ring, 500 13.9 and 20.8; distillation with 16 targets of 160
  // 9.0 and 11.9, of 152 8.5 and 8.0.  (The forms that read a row once need
  // not keep it.)
  if constexpr (MODE == kLossGrad) {
    if (vecs <= 256 * 16 && a.rows > sms)
      return launch_kernel(row_loss_short_kernel<TYPE, OP, MODE, 256, 16>, each, dim3(256), lists,
                           s, a);
  }
  if constexpr (MODE != kLossGrad) {
    int split = 1;
    while (split < kMaxCluster && a.rows * split < int64_t(sms) * kStreamCtas * kStreamWaves &&
           bytes >= split * 2 * kStreamLeast)
      split *= 2;
    while (a.rows * split >= (int64_t(1) << 31)) split /= 2;  // CTA numbers are 31 bits
    return launch_stream<TYPE, OP, MODE>(a, split, lists, s);
  } else {
    return launch_ring<TYPE, OP>(a, sms, bytes, s);
  }
}

}  // namespace lsdrs
