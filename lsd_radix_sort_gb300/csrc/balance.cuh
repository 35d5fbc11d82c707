// K-BALANCE: a router's load-balancing loss, its per-expert counts and the
// gradient.
//
// With p = softmax of a token's scores and c the counts of the expert ids,
// loss = E / (K N^2) sum_e c_e sum_t p_te and
// d loss / d x_tj = E / (K N^2) p_tj (c_j - sum_e c_e p_te): the gradient
// needs the counts of all tokens, but not the probabilities' sums.  So the
// ids (a few words per token) are counted first; then one pass reads each
// token's scores once, adds its probabilities to sums that stay in registers
// (a lane always holds the same experts) and writes its gradient.
//
// A token is held by `group` lanes (a power of two), VECS vectors of WIDTH
// bytes each, so a warp holds 32 / group tokens at a time and one shuffle
// reduces all of them.  Sums over tokens go from lanes to warps and CTAs in
// a fixed order, and from there to the grid as integers (multiples of a power
// of two that the number of tokens sets, fine enough to hold every bit of a
// CTA's sum down to 2^-62 of the total), whose sum does not depend on the
// order: the same bits in every run.
//
// A small call is one cluster that does both steps in one launch and adds up
// through distributed shared memory; a larger one is two launches: the
// counts, one partial histogram per cluster of the first, are added up by
// every CTA of the second.
#pragma once
#include "kernels.h"
#include "losses.h"
#include "scores.cuh"

namespace lsdrs {

// Two CTAs of 8 warps per SM, two tokens per lane under way: with three CTAs,
// one token each, bf16 gradients of 262,144 tokens and 256 experts took 80 us
// instead of 68, with one token and two CTAs 76; lanes per token known at
// compile time took 2 us off that, and a pass among others takes 57 now, the
// counts among them.  42 us is the time of the bytes.  What bounds it is latency: 14.2 instructions per
// score, of which the reductions over a token's lanes are paid per 16 scores,
// at half the issue rate.
constexpr int kBalThreads = 256;
constexpr int kBalCtas = 2;               // per SM
constexpr int kBalWarps = kBalThreads / kWarp;
constexpr int kBalTurns = 4;              // warps that add to one row of sums
constexpr int kBalCluster = 8;            // CTAs of a cluster, at most
constexpr int kBalMaxHists = 19;          // clusters of the counting launch
// Its threads per CTA: their registers leave room for one CTA of the launch
// that comes next, which then has its first scores in L2 when the counts are
// there (bf16 gradients of 262,144 tokens and 256 experts: 57.1 us, 58.1
// without the prefetch; with scores read before the counts 62.4 back to back,
// 65.4 with 1,024 threads here, 65.1 with 256).
constexpr int kCountThreads = 512;
// Scores up to which one cluster does the whole call (8,192 tokens of 64
// experts: 14.6 us in one cluster, 8 in two launches; 32 of 8: 4.8 and 8).
constexpr int64_t kBalSingle = int64_t(1) << 18;

// Scratch: what the counting launch clears (the ticket, a flag for NaN, the
// experts' sums of probabilities), then its clusters' histograms (experts
// counts and the number of tokens each).
struct BalHeader {
  unsigned ticket, nan;
  unsigned long long sums[1];
};
__host__ __device__ constexpr inline size_t bal_header_bytes(int experts) {
  return align_up(static_cast<size_t>(experts) * 8 + 8, 256);
}

__device__ __forceinline__ uint32_t bal_cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t bal_cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void bal_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// A 32-bit word at the same place in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer_word(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Adds the expert ids of tokens first, first + step, ... (threads of the grid
// or the cluster) to hist; hist[experts] counts the tokens that the mask keeps
// (without a mask it is left alone).
__device__ __forceinline__ void count_ids(const BalanceArgs& a, int* hist, int64_t first,
                                          int64_t step) {
  auto add = [&](int64_t e) {
    if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);
  };
  const int64_t n = a.tokens * a.k;
  if (a.mask == nullptr && a.id_stride == a.k &&
      reinterpret_cast<uintptr_t>(a.ids) % 16 == 0) {  // one dense list: 16-byte loads
    const int per = 16 / a.id_bytes;
    const int64_t whole = n / per;
    const uint4* v = static_cast<const uint4*>(a.ids);
    constexpr int kBatch = 8;  // loads under way before the first count
    for (int64_t i = first; i < whole; i += kBatch * step) {
      uint4 w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        w[u] = i + u * step < whole ? __ldcs(v + i + u * step) : make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (a.id_bytes == 8) {
          add(static_cast<int64_t>(static_cast<uint64_t>(w[u].y) << 32 | w[u].x));
          add(static_cast<int64_t>(static_cast<uint64_t>(w[u].w) << 32 | w[u].z));
        } else {
          add(static_cast<int>(w[u].x));
          add(static_cast<int>(w[u].y));
          add(static_cast<int>(w[u].z));
          add(static_cast<int>(w[u].w));
        }
      }
    }
    if (first == 0)
      for (int64_t i = whole * per; i < n; ++i) add(load_index(a.ids, a.id_bytes, i));
    return;
  }
  for (int64_t t = first; t < a.tokens; t += step) {
    if (a.mask != nullptr) {
      if (!a.mask[t]) continue;
      atomicAdd(&hist[a.experts], 1);
    }
    for (int s0 = 0; s0 < a.k; s0 += 8) {  // eight ids under way together
      int64_t e[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        e[u] = s0 + u < a.k ? load_index(a.ids, a.id_bytes, t * a.id_stride + s0 + u) : -1;
#pragma unroll
      for (int u = 0; u < 8; ++u) add(e[u]);
    }
  }
}

// A word at the same place in every CTA of the cluster (0 past its size), all
// of the reads under way together.
__device__ __forceinline__ void peer_words(const void* p, int size, uint32_t (&w)[kBalCluster]) {
#pragma unroll
  for (int r = 0; r < kBalCluster; ++r) w[r] = r < size ? peer_word(p, r) : 0u;
}

// The sum of a word of every CTA's histogram.
__device__ __forceinline__ int cluster_count(const int* hist, int e, int size) {
  uint32_t w[kBalCluster];
  peer_words(hist + e, size, w);
  int n = 0;
#pragma unroll
  for (int r = 0; r < kBalCluster; ++r) n += static_cast<int>(w[r]);
  return n;
}

// WIDTH bytes of scores: as they lie in memory, as floats, and back.
template <int TYPE, int WIDTH>
struct BalVec {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  static constexpr int kN = WIDTH / sizeof(Raw);
  struct alignas(WIDTH) Word {
    Raw r[kN];
  };
  static __device__ __forceinline__ Word load(const Raw* p) {
    Word w;
    if constexpr (WIDTH == 16)
      *reinterpret_cast<uint4*>(&w) = __ldcs(reinterpret_cast<const uint4*>(p));
    else if constexpr (WIDTH == 8)
      *reinterpret_cast<uint2*>(&w) = __ldcs(reinterpret_cast<const uint2*>(p));
    else
      w.r[0] = *p;
    return w;
  }
  static __device__ __forceinline__ Word none() {  // -inf everywhere
    Word w;
#pragma unroll
    for (int i = 0; i < kN; ++i) w.r[i] = static_cast<Raw>(ScoreVec<TYPE>::kMinusInf);
    return w;
  }
  // the largest score of a lane's words; NaN is ignored
  template <int VECS>
  static __device__ __forceinline__ float largest(const Word (&w)[VECS]) {
    float m = -INFINITY;
    if constexpr (sizeof(Raw) == 2 && WIDTH >= 4) {
      uint32_t x = ScoreVec<TYPE>::kMinusInf;
#pragma unroll
      for (int u = 0; u < VECS; ++u)
#pragma unroll
        for (int i = 0; i < WIDTH / 4; ++i)
          x = ScoreVec<TYPE>::larger(x, reinterpret_cast<const uint32_t*>(&w[u])[i]);
      float a, b;
      unpack2(ScoreVec<TYPE>::pair(x), a, b);
      m = fmaxf(a, b);
    } else {
#pragma unroll
      for (int u = 0; u < VECS; ++u)
#pragma unroll
        for (int i = 0; i < kN; ++i) m = fmaxf(m, S::load(w[u].r[i]));
    }
    return m;
  }
  // a lane's words as pairs of floats
  template <int VECS>
  static __device__ __forceinline__ void pairs(const Word (&w)[VECS],
                                               uint64_t (&p)[VECS * kN / 2]) {
#pragma unroll
    for (int j = 0; j < VECS * kN / 2; ++j) {
      const int a = 2 * j, b = 2 * j + 1;
      if constexpr (sizeof(Raw) == 2 && WIDTH >= 4)
        p[j] = ScoreVec<TYPE>::pair(reinterpret_cast<const uint32_t*>(&w[a / kN])[a % kN / 2]);
      else
        p[j] = pack2(S::load(w[a / kN].r[a % kN]), S::load(w[b / kN].r[b % kN]));
    }
  }
  static __device__ __forceinline__ void store(Raw* p, const float (&v)[kN]) {
    Word w;
    if constexpr (sizeof(Raw) == 2 && WIDTH >= 4) {
#pragma unroll
      for (int i = 0; i < WIDTH / 4; ++i)
        reinterpret_cast<uint32_t*>(&w)[i] =
            ScoreVec<TYPE>::word(pack2(v[(2 * i) % kN], v[(2 * i + 1) % kN]));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) w.r[i] = S::store(v[i]);
    }
    if constexpr (WIDTH == 16)
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&w));
    else if constexpr (WIDTH == 8)
      __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(&w));
    else
      *p = w.r[0];
  }
};

// Reductions over the `group` lanes of a token, of several tokens at a time so
// that the shuffles overlap.
template <int N, class F>
__device__ __forceinline__ void group_reduce(float (&v)[N], int group, F&& join) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (group > o) {  // the same for every lane
#pragma unroll
      for (int q = 0; q < N; ++q) v[q] = join(v[q], __shfl_xor_sync(kFull, v[q], o));
    }
  }
}

// out[e] = the sum of n rows of `cols` words, `pitch` words apart, in a fixed
// order.  Where the threads outnumber the columns they share the rows, so that
// the loads are one or two trips to memory; scratch: kBalThreads words.
template <class T>
__device__ __forceinline__ void sum_rows(const T* from, int n, int64_t pitch, int cols, T* out,
                                         T* scratch) {
  const int tid = static_cast<int>(threadIdx.x);
  if (cols > kBalThreads / 2) {
    for (int e = tid; e < cols; e += kBalThreads) {
      T v = 0;
#pragma unroll 8
      for (int r = 0; r < n; ++r) v += __ldcg(from + r * pitch + e);
      out[e] = v;
    }
    __syncthreads();
    return;
  }
  const int teams = kBalThreads / cols, team = tid / cols, e = tid - team * cols;
  if (team < teams) {
    T v = 0;
#pragma unroll 8
    for (int r = team; r < n; r += teams) v += __ldcg(from + r * pitch + e);
    scratch[tid] = v;
  }
  __syncthreads();
  if (tid < cols) {
    T v = 0;
    for (int i = 0; i < teams; ++i) v += scratch[i * cols + tid];
    out[tid] = v;
  }
  __syncthreads();
}

// single: the grid is one cluster, which counts the ids itself.  Otherwise
// `hists` clusters of the counting launch left their histograms in the
// scratch (kLossBwd: the counts are given).
template <int TYPE, int MODE, int WIDTH, int VECS, int GROUP>
__global__ void __launch_bounds__(kBalThreads, kBalCtas)
    balance_kernel(const BalanceArgs a, const int group_, const bool single, const int hists) {
  const int group = GROUP != 0 ? GROUP : group_;
  using B = BalVec<TYPE, WIDTH>;
  using Raw = typename B::Raw;
  constexpr int kN = B::kN;
  // tokens of a lane that are worked on together (as many more are on their way)
  constexpr int kTokens = VECS * kN <= 16 ? 2 : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ bool last;
  __shared__ float warp_part[kBalWarps];
  // share of an expert, E c_e / (K N), laid out so that a warp reads the
  // experts of its lanes without bank conflicts: by fours, the first fours of
  // all vectors before the second ones
  constexpr int kFour = kN < 4 ? 1 : 4, kPlanes = kN / kFour;
  const int all_vecs = VECS * group;
  float* share = reinterpret_cast<float*>(smem);
  auto share_at = [&](int vec, int plane) { return share + (plane * all_vecs + vec) * kFour; };
  int* hist = reinterpret_cast<int*>(share + all_vecs * kN);     // experts + 1
  float* sums = reinterpret_cast<float*>(hist + a.experts + 1);  // kBalWarps / kBalTurns rows
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  const int warp = tid / kWarp;
  const int sub = lane & (group - 1), in_warp = kWarp / group;
  // A warp's tokens: batches of kTokens times in_warp, `step` apart.  The
  // tokens' numbers fit 31 bits; pointers go along.
  const int tokens = static_cast<int>(a.tokens);
  const int64_t step = int64_t(gridDim.x) * kBalWarps * in_warp;
  const int64_t first = (blockIdx.x * int64_t(kBalWarps) + warp) * in_warp + lane / group;
  const Raw* x = static_cast<const Raw*>(a.logits) + first * a.stride + sub * kN;
  Raw* g = static_cast<Raw*>(a.grad) + first * a.grad_stride + sub * kN;
  const int64_t x_step = step * a.stride, g_step = step * a.grad_stride;
  bool on[VECS];  // the lane's vectors that hold experts; the others stay -inf
  typename B::Word raw[kTokens][VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) {
    on[u] = (u * group + sub) * kN < a.experts;
#pragma unroll
    for (int q = 0; q < kTokens; ++q) raw[q][u] = B::none();
  }
  // the batch at t: all of its tokens count (whole), or some may not
  auto load = [&](int64_t t, bool whole) {
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      bool kept = true;
      if (!whole) {
        const int64_t at = t + q * step;
        kept = at < tokens && (a.mask == nullptr || a.mask[at]);
        if (!kept) {  // a token that the mask drops is one without scores
#pragma unroll
          for (int u = 0; u < VECS; ++u) raw[q][u] = B::none();
        }
      }
#pragma unroll
      for (int u = 0; u < VECS; ++u)
        if (kept && on[u]) raw[q][u] = B::load(x + u * group * kN);
      x += x_step;
    }
  };
  // past the last batch of which every lane's tokens exist (the same for the
  // whole warp)
  const int64_t warp_first = first - lane / group;
  const int64_t whole_end =
      a.mask == nullptr ? int64_t(tokens) - (in_warp - 1) - (kTokens - 1) * step : -1;
  // The first batch is on its way while the counts come.  After a counting
  // launch this one may begin before that has ended, and what was queued
  // before it need not be visible yet: until the wait the scores are only
  // brought to L2, where later writes to them are seen too, and read after it.
  // (The backward call has little to wait for: 8.4 us with its loads after the
  // counts for 32,767 f16 tokens of 160 experts, 9.1 before.)
  if (MODE != kLossBwd && !single) {
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
#pragma unroll
      for (int u = 0; u < VECS; ++u)
        if (first + q * step < tokens && on[u]) prefetch_l2(x + q * x_step + u * group * kN);
    }
  }
  grid_dependency_sync();
  if (MODE != kLossBwd) load(first, warp_first < whole_end);

  // ---- the counts
  int tokens_kept;
  if (MODE == kLossBwd) {
    tokens_kept = *a.n_tokens;
    for (int e = tid; e < a.experts; e += kBalThreads) hist[e] = a.counts[e];
  } else if (single) {
    for (int e = tid; e <= a.experts; e += kBalThreads) hist[e] = 0;
    __syncthreads();
    count_ids(a, hist, blockIdx.x * int64_t(kBalThreads) + tid, gridDim.x * int64_t(kBalThreads));
    if (gridDim.x > 1) {
      bal_cluster_sync();
      constexpr int kEach = (RS_MAX_EXPERTS + kBalThreads) / kBalThreads;
      int total[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int e = tid + i * kBalThreads;
        total[i] = e <= a.experts ? cluster_count(hist, e, gridDim.x) : 0;
      }
      bal_cluster_sync();  // every histogram has been read
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (tid + i * kBalThreads <= a.experts) hist[tid + i * kBalThreads] = total[i];
    }
    __syncthreads();
    tokens_kept = a.mask != nullptr ? hist[a.experts] : static_cast<int>(a.tokens);
  } else {
    sum_rows(reinterpret_cast<const int*>(static_cast<unsigned char*>(a.temp) +
                                          bal_header_bytes(a.experts)),
             hists, a.experts + 1, a.experts + 1, hist, reinterpret_cast<int*>(sums));
    tokens_kept = a.mask != nullptr ? hist[a.experts] : static_cast<int>(a.tokens);
  }
  const float n = fmaxf(static_cast<float>(tokens_kept), 1.0f);
  const float each = static_cast<float>(a.experts) / (static_cast<float>(a.k) * n);
  for (int e = tid; e < all_vecs * kN; e += kBalThreads) {
    const bool real = e < a.experts;
    if (MODE != kLossFwd)
      share_at(e / kN, e % kN / kFour)[e % kFour] =
          real ? static_cast<float>(hist[e]) * each : 0.0f;
    if (MODE != kLossBwd && blockIdx.x == 0 && real) a.counts[e] = hist[e];
  }
  if (MODE != kLossBwd && blockIdx.x == 0 && tid == 0) *a.n_tokens = tokens_kept;
  __syncthreads();

  // ---- the tokens
  float scale = a.scale / n;
  if (MODE == kLossBwd && a.grad_loss != nullptr) scale *= *a.grad_loss;
  constexpr int kPairs = VECS * kN / 2;
  uint64_t acc2[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) acc2[j] = 0;
  // the shares of the lane's experts, as pairs (read again for each use: they
  // would take as many registers as the sums)
  auto shares = [&](uint64_t (&w)[kPairs]) {
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      const int vec = u * group + sub;
      if constexpr (kN >= 4) {
#pragma unroll
        for (int h = 0; h < kPlanes; ++h) {
          const float4 q = *reinterpret_cast<const float4*>(share_at(vec, h));
          w[(u * kN + h * 4) / 2] = pack2(q.x, q.y);
          w[(u * kN + h * 4) / 2 + 1] = pack2(q.z, q.w);
        }
      } else if (u % 2 == 0) {
        w[u / 2] = pack2(*share_at(vec, 0), *share_at(vec + group, 0));
      }
    }
  };
  int64_t at = warp_first;
  if (MODE == kLossBwd) load(first, at < whole_end);
  for (; at < tokens; at += step * kTokens) {
    uint64_t v[kTokens][kPairs];
    float m[kTokens], sum[kTokens], dot[kTokens];
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      m[q] = B::largest(raw[q]);
      B::pairs(raw[q], v[q]);
    }
    const int64_t next = at + step * kTokens;
    if (next < tokens) load(next + lane / group, next < whole_end);
    group_reduce(m, group, [](float p, float r) { return fmaxf(p, r); });
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      // exp2(x log2 e - o2), the rounding of o2 (at most 2^5 but for a far
      // origin) being the same for the whole token; f16 has no far scores
      const float o = origin(m[q]);
      float o2 = o * kLog2e, s1 = kLog2e;
      if (TYPE != RS_SCORE_F16 && far_origin(o, o2)) {
        s1 = far_scale(o);
        o2 = o * s1;
      }
      const uint64_t neg_o2 = pack2(-o2, -o2), s2 = pack2(s1, s1);
      uint64_t total = 0, with = 0, sh2[kPairs];
      if (MODE != kLossFwd) shares(sh2);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        v[q][j] = exp2_2(fma2(v[q][j], s2, neg_o2));
        total = add2(total, v[q][j]);
        if (MODE != kLossFwd) with = fma2(v[q][j], sh2[j], with);
      }
      float p0, p1;
      unpack2(total, p0, p1);
      sum[q] = p0 + p1;
      unpack2(with, p0, p1);
      dot[q] = p0 + p1;
    }
    group_reduce(sum, group, [](float p, float r) { return p + r; });
    if (MODE != kLossFwd) group_reduce(dot, group, [](float p, float r) { return p + r; });
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      // 2^-32 <= sum <= 2^32 experts, NaN, or 0 for a token without scores
      const float inv = sum[q] == 0.0f ? 0.0f : __frcp_rn(sum[q]);
      if (MODE != kLossBwd) {
        const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) acc2[j] = fma2(v[q][j], inv2, acc2[j]);
      }
      if (MODE != kLossFwd) {
        // p (share - dot) scale
        const float f = inv * scale, d = dot[q] * inv * f;
        const uint64_t f2 = pack2(f, f), neg_d2 = pack2(-d, -d);
        float y[VECS][kN];
        uint64_t sh2[kPairs];
        shares(sh2);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const int e = 2 * j;
          unpack2(mul2(v[q][j], fma2(sh2[j], f2, neg_d2)), y[e / kN][e % kN],
                  y[(e + 1) / kN][(e + 1) % kN]);
        }
        const bool there = at < whole_end || at + lane / group + q * step < tokens;
#pragma unroll
        for (int u = 0; u < VECS; ++u)
          if (there && on[u]) B::store(g + u * group * kN, y[u]);
        g += g_step;
      }
    }
  }
  float acc[VECS * kN];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) unpack2(acc2[j], acc[2 * j], acc[2 * j + 1]);
  if constexpr (MODE != kLossBwd) {
    // ---- the sums over tokens
#pragma unroll
    for (int j = 0; j < VECS * kN; ++j)
      for (int o = group; o < kWarp; o <<= 1) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
    constexpr int kRows = kBalWarps / kBalTurns;
    for (int turn = 0; turn < kBalTurns; ++turn) {
      if (warp / kRows == turn && lane < group) {
        float* row = sums + (warp % kRows) * a.experts;
#pragma unroll
        for (int u = 0; u < VECS; ++u)
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int e = (u * group + sub) * kN + i;
            if (e < a.experts) row[e] = turn == 0 ? acc[u * kN + i] : row[e] + acc[u * kN + i];
          }
      }
      __syncthreads();
    }
    for (int e = tid; e < a.experts; e += kBalThreads) {
      float p = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) p += sums[r * a.experts + e];
      sums[e] = p;
    }
    float loss = 0.0f;
    if (single) {
      const int size = static_cast<int>(gridDim.x);
      if (size > 1)
        bal_cluster_sync();
      else
        __syncthreads();
      if (blockIdx.x == 0) {  // the first CTA adds up, in rank order
        for (int e = tid; e < a.experts; e += kBalThreads) {
          uint32_t w[kBalCluster];
          peer_words(sums + e, size, w);
          float p = 0.0f;
#pragma unroll
          for (int r = 0; r < kBalCluster; ++r) p += __uint_as_float(w[r]);
          p /= n;
          a.mean_probs[e] = p;
          loss += static_cast<float>(hist[e]) * each * p;
        }
      }
      if (size > 1) bal_cluster_sync();  // no CTA ends while its sums are read
      if (blockIdx.x != 0) return;
    } else {
      __syncthreads();
      BalHeader* to = static_cast<BalHeader*>(a.temp);
      // p <= tokens < 2^bits, so sums of p 2^shift stay below 2^62
      const int shift = 62 - (32 - __clz(tokens_kept | 1));
      const float up = ldexpf(1.0f, shift);
      bool nan = false;
      for (int e = tid; e < a.experts; e += kBalThreads) {
        const float p = sums[e];
        if (isnan(p))
          nan = true;
        else
          atomicAdd(&to->sums[e], static_cast<unsigned long long>(__float2ll_rn(p * up)));
      }
      if (nan) atomicOr(&to->nan, 1u);
      __threadfence();
      __syncthreads();
      if (tid == 0) last = atomicAdd(&to->ticket, 1u) == gridDim.x - 1;
      __syncthreads();
      if (!last) return;
      __threadfence();
      const bool any_nan = __ldcg(&to->nan) != 0;
      for (int e = tid; e < a.experts; e += kBalThreads) {
        const float total = __ull2float_rn(__ldcg(&to->sums[e]));
        const float p = any_nan ? NAN : total / up / n;
        a.mean_probs[e] = p;
        loss += static_cast<float>(hist[e]) * each * p;
      }
    }
    loss = warp_sum(loss);
    if (lane == 0) warp_part[warp] = loss;
    __syncthreads();
    if (tid == 0) {
      loss = 0.0f;
      for (int i = 0; i < kBalWarps; ++i) loss += warp_part[i];
      *a.loss = loss;
    }
  }
}

inline size_t bal_smem(int experts) {
  const size_t sums = static_cast<size_t>(experts) * (kBalWarps / kBalTurns);
  // the shares are padded to whole lanes: up to 32 of up to 32 scores
  return (size_t(RS_MAX_EXPERTS) + experts + 1 + (sums > kBalThreads ? sums : kBalThreads)) * 4;
}

template <int TYPE, int MODE, int WIDTH, int VECS, int GROUP>
cudaError_t launch_balance_shape(const BalanceArgs& a, int group, bool single, int ctas,
                                 int cluster, int hists, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kBalThreads);
  cfg.dynamicSmemBytes = bal_smem(a.experts);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
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
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, balance_kernel<TYPE, MODE, WIDTH, VECS, GROUP>, a, group, single,
                            hists);
}

cudaError_t launch_balance_counts(const BalanceArgs& a, int clusters, cudaStream_t s);

template <int TYPE, int MODE>
cudaError_t launch_balance_as(const BalanceArgs& a, int* launched, cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<TYPE>::Raw);
  auto multiple = [&](int bytes) {
    return reinterpret_cast<uintptr_t>(a.logits) % bytes == 0 && a.stride * kEs % bytes == 0 &&
           a.experts * kEs % bytes == 0 &&
           (MODE == kLossFwd || (reinterpret_cast<uintptr_t>(a.grad) % bytes == 0 &&
                                 a.grad_stride * kEs % bytes == 0));
  };
  const int width = multiple(16) ? 16 : kEs == 2 && multiple(8) ? 8 : kEs;
  const int per = width / kEs, vecs = (a.experts + per - 1) / per;
  // vectors per lane: up to 32 scores; the least idle lanes, and among equals
  // the fewest vectors that make 8 scores a lane and at most 16 lanes a token
  // (more lanes cost more shuffles per score, more scores a lane leave fewer
  // tokens under way; 64 to 256 experts measured 10 to 40% apart)
  int best = 0, group = 32;
  double waste = 1e30;
  bool fits = false;
  for (int v : {1, 2, 4, 8, 16, 32}) {
    if (v * per > 32 || (per == 1 && v != 2 && v != 8 && v != 32)) continue;
    int g = 1;
    while (g < 32 && g * v < vecs) g *= 2;
    if (g * v < vecs) continue;
    const double w = static_cast<double>(g) * v / vecs;
    if (w < waste - 1e-9 || (w < waste + 1e-9 && !fits)) {
      waste = w;
      best = v;
      group = g;
      fits = v * per >= 8 && g <= 16;
    }
  }
  if (best == 0) return cudaErrorInvalidValue;
  // how the work is cut
  const int in_cta = kBalWarps * (kWarp / group);
  const int64_t ctas_for = (a.tokens + in_cta - 1) / in_cta;
  bool single = false;
  int ctas, cluster = 1, hists = 0;
  if (MODE == kLossBwd) {
    const int64_t most = int64_t(device_sm_count()) * 4;
    ctas = static_cast<int>(ctas_for < most ? ctas_for : most);
  } else if (a.tokens * a.experts <= kBalSingle) {
    single = true;
    while (cluster < kBalCluster && cluster < ctas_for) cluster *= 2;
    ctas = cluster;
  } else {
    // a warp takes two batches at least before there is another CTA
    const int64_t most = int64_t(device_sm_count()) * kBalCtas, half = (ctas_for + 1) / 2;
    ctas = static_cast<int>(half < 1 ? 1 : half < most ? half : most);
    const int64_t each = int64_t(kCountThreads) * kBalCluster * 4;
    const int64_t want = (a.tokens * a.k + each - 1) / each;
    hists = static_cast<int>(want < 1 ? 1 : want < kBalMaxHists ? want : kBalMaxHists);
    const cudaError_t e = launch_balance_counts(a, hists, s);
    if (e != cudaSuccess) return e;
    *launched = 2;
  }
  // the lanes per token are known at compile time for 16-byte vectors
  auto shape = [&](auto w, auto v, auto g) {
    return launch_balance_shape<TYPE, MODE, decltype(w)::value, decltype(v)::value,
                                decltype(g)::value>(a, group, single, ctas, cluster, hists, s);
  };
  auto go = [&](auto w, auto v) { return shape(w, v, ScoreTag<0>{}); };
  auto wide = [&](auto v) {
    if (group == 8) return shape(ScoreTag<16>{}, v, ScoreTag<8>{});
    if (group == 16) return shape(ScoreTag<16>{}, v, ScoreTag<16>{});
    return go(ScoreTag<16>{}, v);
  };
  constexpr int k4 = 4 / kEs;  // 16-byte vectors hold half as many 32-bit scores
  if (width == 16) {
    if (best == 1) return wide(ScoreTag<1>{});
    if (best == 2) return wide(ScoreTag<2>{});
    if (best == 4) return wide(ScoreTag<4>{});
    if constexpr (k4 == 1)
      if (best == 8) return go(ScoreTag<16>{}, ScoreTag<8>{});
  } else if (width == kEs) {
    if (best == 2) return go(ScoreTag<kEs>{}, ScoreTag<2>{});
    if (best == 8) return go(ScoreTag<kEs>{}, ScoreTag<8>{});
    if (best == 32) return go(ScoreTag<kEs>{}, ScoreTag<32>{});
  } else if constexpr (kEs == 2) {
    if (best == 1) return go(ScoreTag<8>{}, ScoreTag<1>{});
    if (best == 2) return go(ScoreTag<8>{}, ScoreTag<2>{});
    if (best == 4) return go(ScoreTag<8>{}, ScoreTag<4>{});
    if (best == 8) return go(ScoreTag<8>{}, ScoreTag<8>{});
  }
  return cudaErrorInvalidValue;
}

template <int TYPE>
cudaError_t launch_balance_of(LossMode mode, const BalanceArgs& a, int* launched, cudaStream_t s) {
  switch (mode) {
    case kLossFwd: return launch_balance_as<TYPE, kLossFwd>(a, launched, s);
    case kLossGrad: return launch_balance_as<TYPE, kLossGrad>(a, launched, s);
    case kLossBwd: return launch_balance_as<TYPE, kLossBwd>(a, launched, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lsdrs
