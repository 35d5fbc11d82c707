// K-LOGPROBS: the log probabilities of given tokens, the entropy and the top
// alternatives of rows of logits, and the gradient of all of them.
//
// With y_j = (x_j - m) / t, e_j = exp y_j, S = sum e_j and m the largest score
// of a row:  logp_j = y_j - log S,  H = log S - sum e_j y_j / S.  S and the
// entropy's sum are taken in one pass, both moved along whenever the origin
// of the exponents moves.
#pragma once
#include "row_loss.cuh"
#include "vocab.h"

namespace lsdrs {

// ------------------------------------------------------------------ statistics
// A softmax in progress with its entropy's sum: m the largest score, sum =
// sum e, dot = sum e y with y in units of log 2.
struct Stats {
  float m, sum, dot;
};

// An exponent that says 2^x = 0 and can still be multiplied by 0.
constexpr float kNothing = -256.0f;
__device__ __forceinline__ float above_nothing(float y) {  // NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(kNothing));
  return r;
}

// The same taken from another origin, d = (old - new) scale below or above it.
__device__ __forceinline__ Stats moved(const Stats& s, float m, float d) {
  d = fmaxf(d, kNothing);  // (what is that far below is 0)
  const float w = exp2_approx(d);
  return {m, s.sum * w, w * (s.dot + d * s.sum)};
}

__device__ __forceinline__ Stats warp_join(const Stats& v, float scale2) {
  const float m = warp_max(v.m);
  const Stats s = moved(v, m, (v.m - origin(m)) * scale2);
  return {m, warp_sum(s.sum), warp_sum(s.dot)};
}

// A thread's part of it over many vectors; like RunningSoftmax, with the
// products of the exponentials and their exponents as well.
template <int TYPE>
struct RunningStats {
  float scale, slack, o, limit, top;
  Exponent e;
  uint64_t sum[2], dot[2];

  __device__ __forceinline__ explicit RunningStats(float scale2)
      : scale(scale2),
        slack(8.0f / scale2),
        o(-INFINITY),
        limit(-INFINITY),
        top(-INFINITY),
        e(0.0f, scale2) {
    sum[0] = sum[1] = dot[0] = dot[1] = 0;
  }
  // what the exponents lack because e.os2 is rounded, e.mend = 2^lack
  __device__ __forceinline__ float lack() const {
    return o == -INFINITY ? 0.0f : __fmaf_rn(-o, e.scale, e.os2);
  }
  __device__ __forceinline__ Stats at_origin() const {
    float a, b, c, d;
    unpack2(add2(sum[0], sum[1]), a, b);
    unpack2(add2(dot[0], dot[1]), c, d);
    return {o, (a + b) * e.mend, (c + d + lack() * (a + b)) * e.mend};
  }
  __device__ __forceinline__ void move(float m) {
    const Stats s = moved(at_origin(), m, (o - m) * scale);
    o = m;
    limit = m + slack;
    e = Exponent(m, scale);
    const float a = __fdividef(s.sum, e.mend);
    sum[0] = pack2(a, 0.0f);
    dot[0] = pack2(__fdividef(s.dot, e.mend) - lack() * a, 0.0f);
    sum[1] = dot[1] = 0;
  }
  // Adds vectors; returns their largest score.
  template <int VECS>
  __device__ __forceinline__ float add(const uint4 (&v)[VECS]) {
    const float m = vec_max<TYPE>(v);
    top = fmaxf(top, m);
    if (m > limit) move(m);
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      uint64_t p[ScoreVec<TYPE>::kCount / 2];
      vec_pairs<TYPE>(v[u], p);
#pragma unroll
      for (int i = 0; i < ScoreVec<TYPE>::kCount / 2; ++i) {
        float a, b;
        unpack2(fma2(p[i], pack2(e.scale, e.scale), pack2(-e.os2, -e.os2)), a, b);
        const uint64_t y = pack2(above_nothing(a), above_nothing(b));
        const uint64_t x = exp2_2(y);
        sum[i & 1] = add2(sum[i & 1], x);
        dot[i & 1] = fma2(x, y, dot[i & 1]);
      }
    }
    return m;
  }
  __device__ __forceinline__ Stats result() const {
    const Stats s = at_origin();
    return top > o ? moved(s, top, (o - top) * scale) : s;
  }
};

// ------------------------------------------------------------ top alternatives
// Scores as unsigned integers in their order, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kOrderLeast = 0x00800000u;  // of the lowest finite score

// A score and its column in one word: the larger word is the better score, of
// equal ones the one of the lower column.
__device__ __forceinline__ uint64_t entry_of(uint32_t order, int col) {
  return static_cast<uint64_t>(order) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ uint32_t entry_order(uint64_t e) { return static_cast<uint32_t>(e >> 32); }
__device__ __forceinline__ int entry_col(uint64_t e) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(e));
}

constexpr int kLpThreads = kStreamThreads;
constexpr int kLpWarps = kLpThreads / kWarp;
constexpr int kLpCtas = 3;      // per SM
constexpr int kLpSlots = 32;    // maxima that a thread keeps of its vectors
constexpr int kLpRadix = 256;
constexpr int kLpCounted = 128; // candidates whose ranks are counted, not sorted
constexpr int64_t kLpLists = 4096;  // entries that a cluster exchanges at most

// Candidates held of a segment.
__host__ __device__ constexpr inline int candidate_room(int top) { return top <= 128 ? 512 : 2048; }

// Shared memory behind the static part: candidates, the cluster's lists, and
// every thread's maxima.
__host__ __device__ constexpr inline size_t logprobs_smem(int top, int split, int slots) {
  return top == 0 ? 0
                  : static_cast<size_t>(candidate_room(top)) * 8 +
                        (split > 1 ? static_cast<size_t>(split) * top * 8 : 0) +
                        static_cast<size_t>(slots) * kLpThreads * 2;
}

struct alignas(16) TopShared {
  uint32_t tops[kLpThreads];     // largest scores of groups of threads
  uint32_t hist[kLpRadix];
  uint32_t least;                // no candidate is below this
  int count;                     // candidates
  uint64_t prefix;               // exact selection: entries from here on are kept,
  int above, reach;              // so many are above its digits, at or above them
};

// A CTA's segment of a row as its threads have read it: every thread's
// vectors begin + tid + i * kLpThreads in batches, 2^shift batches to a slot
// of which it has kept the largest score (as the upper half of its order).
template <int TYPE>
struct Segment {
  using Raw = typename Score<TYPE>::Raw;
  const Raw* x;
  const RowVecs<TYPE>& vecs;
  int begin, end, shift, slots;
  const uint16_t* kept;

  // f(order, column) for this thread's scores of slots that reach `least`
  template <class F>
  __device__ __forceinline__ void each(uint32_t least, F&& f) const {
    constexpr int kN = ScoreVec<TYPE>::kCount;
    const int tid = static_cast<int>(threadIdx.x);
    const uint4* xv = reinterpret_cast<const uint4*>(x - vecs.lead);
    uint32_t hit = 0;
    for (int s = 0; s < slots; ++s)
      hit |= static_cast<uint32_t>(kept[s * kLpThreads + tid] >= least >> 16) << s;
    while (hit != 0) {
      const int s = __ffs(static_cast<int>(hit)) - 1;
      hit &= hit - 1;
      const int64_t first = begin + tid + (static_cast<int64_t>(s) << shift) * Stream<TYPE>::kStep;
      const int64_t last =
          min(static_cast<int64_t>(end),
              first + (static_cast<int64_t>(Stream<TYPE>::kStep) << shift));
      for (int64_t v0 = first; v0 < last; v0 += Stream<TYPE>::kStep) {
        uint4 r[kStreamBatch];
#pragma unroll
        for (int u = 0; u < kStreamBatch; ++u) {
          const int64_t v = v0 + u * kLpThreads;
          constexpr uint32_t kNone = ScoreVec<TYPE>::kMinusInf;
          r[u] = v < last ? vecs.load(xv, x, static_cast<int>(v))
                          : make_uint4(kNone, kNone, kNone, kNone);
        }
#pragma unroll
        for (int u = 0; u < kStreamBatch; ++u) {
          const uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
          const int col = static_cast<int>((v0 + u * kLpThreads) * kN - vecs.lead);
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const Raw raw = static_cast<Raw>(kN == 4 ? w[i & 3] : w[i >> 1] >> (16 * (i & 1)));
            const uint32_t o = order_of(Score<TYPE>::load(raw));
            if (o >= least) f(o, col + i);
          }
        }
      }
    }
  }
};

// Adds to a histogram; lanes with the same digit at once.
__device__ __forceinline__ void count_digit(uint32_t* hist, uint32_t digit) {
  const unsigned active = __activemask();
  const unsigned same = __match_any_sync(active, digit);
  if (lane_id() == static_cast<uint32_t>(__ffs(static_cast<int>(same)) - 1))
    atomicAdd(&hist[digit], static_cast<uint32_t>(__popc(same)));
}

// More candidates than there is room for (many equal scores, or a long list):
// entries are narrowed down digit by digit, 8 bits from the top, by counting
// those that share the digits so far, until what is at and above them fits.
// Entries differ, so they do at last.
template <int TYPE>
__device__ __noinline__ void select_exactly(const Segment<TYPE>& seg, int top, int room,
                                            TopShared* sh, uint64_t* cand) {
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t least = sh->least;
  uint64_t prefix = 0;  // entries at or above it are kept, those of its digits divided further
  int shift = 64, above = 0;
  do {
    shift -= 8;
    for (int i = tid; i < kLpRadix; i += kLpThreads) sh->hist[i] = 0;
    __syncthreads();
    seg.each(least, [&](uint32_t o, int col) {
      const uint64_t e = entry_of(o, col);
      if (shift == 56 || (e ^ prefix) >> (shift + 8) == 0)
        count_digit(sh->hist, static_cast<uint32_t>(e >> shift) & 0xFFu);
    });
    __syncthreads();
    if (tid == 0) {
      int n = above, d = kLpRadix - 1;
      while (d > 0 && n + static_cast<int>(sh->hist[d]) < top) n += static_cast<int>(sh->hist[d--]);
      sh->prefix = prefix | static_cast<uint64_t>(d) << shift;
      sh->above = n;
      sh->reach = n + static_cast<int>(sh->hist[d]);
    }
    __syncthreads();
    prefix = sh->prefix;
    above = sh->above;
  } while (sh->reach > room && shift > 0);
  if (tid == 0) sh->count = 0;
  __syncthreads();
  seg.each(least, [&](uint32_t o, int col) {
    const uint64_t e = entry_of(o, col);
    if (e >= prefix) {
      const int at = atomicAdd(&sh->count, 1);
      if (at < room) cand[at] = e;
    }
  });
  __syncthreads();
}

// Sorts n entries, the largest first; room for the next power of two.
static __device__ __noinline__ void sort_entries(uint64_t* e, int n) {
  const int tid = static_cast<int>(threadIdx.x);
  int size = 2;
  while (size < n) size *= 2;
  for (int i = n + tid; i < size; i += kLpThreads) e[i] = 0;
  __syncthreads();
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      for (int p = tid; p < size / 2; p += kLpThreads) {
        const int i = (p & ~(step - 1)) * 2 + (p & (step - 1)), j = i + step;
        const uint64_t a = e[i], b = e[j];
        if ((a < b) == ((i & run) == 0)) {
          e[i] = b;
          e[j] = a;
        }
      }
      __syncthreads();
    }
}

__device__ __forceinline__ void store_peer(uint64_t* at, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(peer_addr(smem_addr(at), rank)), "l"(v)
               : "memory");
}
__device__ __forceinline__ void store_peer(Stats* at, uint32_t rank, const Stats& v) {
  const uint32_t to = peer_addr(smem_addr(at), rank);
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v.m) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(v.sum) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(v.dot) : "memory");
}

// What the outputs of a row are computed from.
struct RowStats {
  float m, log_sum, entropy;
  bool nan, empty;

  __device__ __forceinline__ explicit RowStats(const Stats& s)
      : m(s.m), log_sum(logf(s.sum)), nan(isnan(s.sum)), empty(s.sum == 0.0f) {
    constexpr float kLn2 = 0.69314718055994531f;
    entropy = empty ? 0.0f : log_sum - kLn2 * (s.dot / s.sum);
  }
  __device__ __forceinline__ float logprob(float x, float tau) const {
    // halves: a difference of two finite scores may be more than a float holds
    return nan ? NAN : empty ? -INFINITY : (0.5f * x - 0.5f * m) / (0.5f * tau) - log_sum;
  }
};

__device__ __forceinline__ void store_top(const LogprobArgs& a, int64_t row, int at, uint64_t e,
                                          const RowStats& s) {
  a.top_logprobs[row * a.top + at] =
      s.nan ? NAN : s.logprob(score_of(entry_order(e)), a.tau);
  a.top_ids[row * a.top + at] = s.nan ? -1 : entry_col(e);
}

// One CTA, or a cluster of `split`, per row.  Its scores pass through once
// (batches of 4 vectors per thread, the next one under way); the top
// alternatives cost that pass nothing but a maximum per batch, which it needs
// anyway: a slot per thread and some batches keeps it.  Afterwards the
// largest scores of 64 to 256 groups of threads give a bound: `top` of them
// reach it, so no score below it can be among the `top` best, and few others
// reach it (of 64 groups about 24 scores for the best 20).  Only the batches
// whose maximum reaches the bound are read again, from L2.
template <int TYPE>
__global__ void __launch_bounds__(kLpThreads, kLpCtas)
    logprobs_kernel(const __grid_constant__ LogprobArgs a, const int split, const int slots,
                    const int shift) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Stats part[kLpWarps], peer[kMaxCluster];
  __shared__ TopShared sh;
  __shared__ int lengths[kMaxCluster];
  const int top = a.top, room = candidate_room(top);
  uint64_t* cand = reinterpret_cast<uint64_t*>(smem);
  uint64_t* lists = cand + room;  // the cluster's, `top` entries each
  uint16_t* kept = reinterpret_cast<uint16_t*>(lists + (split > 1 ? split * top : 0));
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int lane = static_cast<int>(lane_id());
  grid_dependency_sync();
  if (split > 1) cluster_begun();
  const int64_t row = blockIdx.x / split;
  const int rank = static_cast<int>(blockIdx.x % split);
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  const RowVecs<TYPE> vecs(x, static_cast<int>(a.cols));
  const int per = (vecs.count + split - 1) / split;
  const int begin = min(rank * per, vecs.count), end = min(begin + per, vecs.count);
  const float scale2 = a.scale2;

  // the first tokens' scores, under way with the row's
  float x0 = 0.0f;
  bool live0 = false;
  if (rank == 0 && tid < a.k) {
    const int64_t i = load_index(a.tokens, a.index_bytes, row * a.token_stride + tid);
    live0 = i >= 0 && i < a.cols;
    if (live0) x0 = S::load(x[i]);
  }
  RunningStats<TYPE> run(scale2);
  Stream<TYPE> stream(x, vecs, begin, end, tid);
  if (top == 0) {
    stream.run([&](int, const uint4(&r)[kStreamBatch]) { run.add(r); });
  } else {
    for (int s = 0; s < slots; ++s) kept[s * kLpThreads + tid] = 0;
    int batch = 0;
    float m = -INFINITY;
    stream.run([&](int, const uint4(&r)[kStreamBatch]) {
      m = fmaxf(m, run.add(r));
      if ((++batch & ((1 << shift) - 1)) == 0) {
        kept[((batch - 1) >> shift) * kLpThreads + tid] =
            static_cast<uint16_t>(order_of(m) >> 16);
        m = -INFINITY;
      }
    });
    if ((batch & ((1 << shift) - 1)) != 0)
      kept[(batch >> shift) * kLpThreads + tid] = static_cast<uint16_t>(order_of(m) >> 16);
  }
  Stats s = warp_join(run.result(), scale2);
  if (lane == 0) part[warp] = s;

  if (top > 0) {
    // the bound: of 64, 128 or 256 groups the `top`-th largest maximum; in
    // each group's order the last 8 bits make room for its number
    const int fold = top <= 32 ? 4 : top <= 64 ? 2 : 1, groups = kLpThreads / fold;
    float g = run.top;
    if (fold > 1) g = fmaxf(g, __shfl_xor_sync(kFull, g, 1));
    if (fold > 2) g = fmaxf(g, __shfl_xor_sync(kFull, g, 2));
    if (tid % fold == 0) sh.tops[tid / fold] = (order_of(g) & ~0xFFu) | (tid / fold);
    if (tid == 0) {
      sh.count = 0;
      sh.least = kOrderLeast;  // stays where the groups are too few, or -inf
    }
    __syncthreads();
    if (top <= groups / 2 && tid < groups) {
      const uint32_t own = sh.tops[tid];
      int better = 0;
      for (int i = 0; i < groups; i += 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(&sh.tops[i]);
        better += (t.x > own) + (t.y > own) + (t.z > own) + (t.w > own);
      }
      if (better == top - 1) sh.least = max(own & ~0xFFu, kOrderLeast);
    }
  }
  __syncthreads();
  s = warp_join(lane < kLpWarps ? part[lane] : Stats{-INFINITY, 0.0f, 0.0f}, scale2);

  int found = 0;
  if (top > 0) {
    const Segment<TYPE> seg{x, vecs, begin, end, shift, slots, kept};
    seg.each(sh.least, [&](uint32_t o, int col) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < room) cand[at] = entry_of(o, col);
    });
    __syncthreads();
    if (sh.count > room) select_exactly<TYPE>(seg, top, room, &sh, cand);
    found = min(sh.count, room);
  }
  if (split > 1) {
    cluster_wait();  // all CTAs of the cluster have begun
    if (tid < split) {
      store_peer(&peer[rank], tid, s);
      store_peer(&lengths[rank], tid, min(found, top));
    }
  }
  const RowStats alone(s);
  // of the segment's candidates the best go to the row's list, or every CTA's
  auto place = [&](int at, uint64_t e) {
    if (at >= top) return;
    if (split == 1)
      store_top(a, row, at, e, alone);
    else
      for (int r = 0; r < split; ++r) store_peer(&lists[rank * top + at], r, e);
  };
  if (found <= kLpCounted) {
    if (tid < found) {
      const uint64_t e = cand[tid];
      int better = 0;
      for (int i = 0; i < found; ++i) better += cand[i] > e;
      place(better, e);
    }
  } else {
    sort_entries(cand, found);
    for (int i = tid; i < found; i += kLpThreads) place(i, cand[i]);
  }
  int total = found;
  if (split > 1) {
    cluster_sync();
    s = warp_join(lane < split ? peer[lane] : Stats{-INFINITY, 0.0f, 0.0f}, scale2);
    total = 0;
    for (int r = 0; r < split; ++r) total += lengths[r];
  }
  const RowStats st(s);
  if (split > 1 && top > 0) {
    // an entry's place: those above it in each CTA's list, which is in order
    const int mine = min(found, top);
    for (int first = 0; first < mine; first += kLpThreads) {
      const int n = min(mine - first, kLpThreads);
      if (tid < n) sh.hist[tid] = 0;
      __syncthreads();
      for (int p = tid; p < n * split; p += kLpThreads) {
        const int i = p / split, r = p % split;
        const uint64_t e = lists[rank * top + first + i];
        const uint64_t* list = lists + r * top;
        int lo = 0, hi = lengths[r];
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (list[mid] > e)
            lo = mid + 1;
          else
            hi = mid;
        }
        if (lo > 0) atomicAdd(&sh.hist[i], static_cast<uint32_t>(lo));
      }
      __syncthreads();
      if (tid < n && sh.hist[tid] < static_cast<uint32_t>(top))
        store_top(a, row, static_cast<int>(sh.hist[tid]), lists[rank * top + first + tid], st);
      __syncthreads();
    }
  }
  if (rank != 0) return;
  for (int i = total + tid; i < top; i += kLpThreads) {  // fewer scores than asked for
    a.top_logprobs[row * top + i] = st.nan ? NAN : -INFINITY;
    a.top_ids[row * top + i] = -1;
  }
  if (tid < a.k) a.logprobs[row * a.k + tid] = live0 ? st.logprob(x0, a.tau) : 0.0f;
  for (int i = tid + kLpThreads; i < a.k; i += kLpThreads) {
    const int64_t c = load_index(a.tokens, a.index_bytes, row * a.token_stride + i);
    a.logprobs[row * a.k + i] =
        c >= 0 && c < a.cols ? st.logprob(S::load(x[c]), a.tau) : 0.0f;
  }
  if (tid == 0) {
    a.entropy[row] = st.entropy;
    a.lse[row] = st.nan ? NAN : st.empty ? -INFINITY : st.m / a.tau + st.log_sum;
    a.stats[row] = make_float2(st.nan ? NAN : st.m, st.log_sum);
  }
}

// -------------------------------------------------------------------- backward
// With s the sum of the upstream gradients of a row's tokens and alternatives,
//
//   t dx_j = q_j (g_lse - s - g_H (log q_j + H)) + sum over entries of column j
//
// that is 2^y_j (c0 + c1 y_j) with y_j the exponent from the row's maximum, in
// units of log 2: two multiply-adds and one exponential per score.  The
// entries' columns are written last.
struct Pull {
  float c0, c1;
};

template <int TYPE>
__global__ void __launch_bounds__(kLpThreads, kLpCtas)
    logprobs_backward_kernel(const __grid_constant__ LogprobArgs a, const int split,
                             const bool together) {
  using S = Score<TYPE>;
  using Raw = typename S::Raw;
  using V = ScoreVec<TYPE>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float warp_part[kLpWarps];
  grid_dependency_sync();
  // the entries: columns (-1: none), upstream gradients, scores
  const int n = (a.grad_logprobs != nullptr ? a.k : 0) + (a.grad_top != nullptr ? a.top : 0);
  const int n_tokens = a.grad_logprobs != nullptr ? a.k : 0;
  int* col = reinterpret_cast<int*>(smem);
  float* up = reinterpret_cast<float*>(col + n);
  float* score = up + n;
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int lane = static_cast<int>(lane_id());
  const int64_t row = blockIdx.x / split;
  const int rank = static_cast<int>(blockIdx.x % split);
  const Raw* x = static_cast<const Raw*>(a.logits) + row * a.stride;
  Raw* g = static_cast<Raw*>(a.grad) + row * a.grad_stride;
  const RowVecs<TYPE> vecs(x, static_cast<int>(a.cols));
  const int per = (vecs.count + split - 1) / split;
  const int begin = min(rank * per, vecs.count), end = min(begin + per, vecs.count);
  const RowOut<TYPE> out(g, vecs);
  Stream<TYPE> stream(x, vecs, begin, end, tid);  // the first loads are under way
  const float2 stats = a.stats[row];
  const float entropy = a.entropy != nullptr ? a.entropy[row] : 0.0f;
  const float g_entropy = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.0f;
  const float g_lse = a.grad_lse != nullptr ? a.grad_lse[row] : 0.0f;
  float sum = 0.0f;
  for (int i = tid; i < n; i += kLpThreads) {
    const bool token = i < n_tokens;
    const int64_t c = token ? load_index(a.tokens, a.index_bytes, row * a.token_stride + i)
                            : a.top_ids[row * a.top + i - n_tokens];
    const bool live = c >= 0 && c < a.cols;
    const float u = !live   ? 0.0f
                    : token ? a.grad_logprobs[row * a.k + i]
                            : a.grad_top[row * a.top + i - n_tokens];
    col[i] = live ? static_cast<int>(c) : -1;
    up[i] = u;
    score[i] = live ? S::load(x[c]) : 0.0f;
    sum += u;
  }
  sum = warp_sum(sum);
  if (lane == 0) warp_part[warp] = sum;
  __syncthreads();
  sum = warp_sum(lane < kLpWarps ? warp_part[lane] : 0.0f);
  // an empty row (no score above -inf) has no gradient
  const bool empty = stats.x == -INFINITY;
  const float m = empty ? 0.0f : stats.x;
  const Exponent e(m, a.scale2);
  const float lack = __fmaf_rn(-m, e.scale, e.os2);
  const float log2_sum = stats.y * kLog2e;
  constexpr float kLn2 = 0.69314718055994531f;
  const float f = empty ? 0.0f : expf(-stats.y) * e.mend * a.inv_tau;
  const float b = -g_entropy * kLn2;
  Pull pull;
  pull.c1 = empty ? 0.0f : f * b;
  pull.c0 = empty ? 0.0f : f * (g_lse - sum - g_entropy * entropy + b * (lack - log2_sum));
  const bool nothing = pull.c0 == 0.0f && pull.c1 == 0.0f;
  // over its own logits no CTA of the row may write before all of them have
  // read the entries' scores
  if (together) cluster_sync();
  const int inner_end = min(end, vecs.whole_end());
  auto put = [&](int v0, const uint4(&r)[kStreamBatch]) {
    const int first = v0 - lane;  // the same for all lanes of the warp
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
  if (nothing) {  // the row's scores do not matter
    const uint4 zero[kStreamBatch] = {};
    for (int v = begin + tid; v < end; v += kStreamThreads * kStreamBatch) put(v, zero);
  } else {
    const uint64_t c0 = pack2(pull.c0, pull.c0), c1 = pack2(pull.c1, pull.c1);
    stream.run([&](int v, uint4(&r)[kStreamBatch]) {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) {
        uint64_t p[V::kCount / 2];
        vec_pairs<TYPE>(r[u], p);
#pragma unroll
        for (int i = 0; i < V::kCount / 2; ++i) {
          float y0, y1;
          unpack2(fma2(p[i], pack2(e.scale, e.scale), pack2(-e.os2, -e.os2)), y0, y1);
          const uint64_t y = pack2(above_nothing(y0), above_nothing(y1));
          p[i] = mul2(exp2_2(y), fma2(c1, y, c0));
        }
        r[u] = vec_of<TYPE>(p);
      }
      put(v, r);
    });
  }
  if (n == 0) return;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(begin) * V::kCount - vecs.lead;
  const int64_t last = static_cast<int64_t>(end) * V::kCount - vecs.lead;
  for (int i = tid; i < n; i += kLpThreads) {
    const int c = col[i];
    if (c < 0 || c < first || c >= last) continue;
    // a column named more than once: its first entry writes, for all of them
    bool mine = true;
    float total = 0.0f;
    for (int j = 0; j < n && mine; ++j) {
      if (col[j] != c) continue;
      mine = j >= i;
      total += up[j];
    }
    if (!mine) continue;
    const float y = above_nothing(__fmaf_rn(score[i], e.scale, -e.os2));
    g[c] = S::store(exp2_approx(y) * __fmaf_rn(pull.c1, y, pull.c0) +
                    (empty ? 0.0f : total * a.inv_tau));
  }
}

// ---------------------------------------------------------------------- launch
constexpr int kLpMaxSmem = 65536;  // candidates, lists and maxima at their most
static_assert(logprobs_smem(1024, static_cast<int>(kLpLists) / 1024, kLpSlots) <= kLpMaxSmem);

// Opts a kernel into its dynamic shared memory and clusters of 16, once per
// device.
template <class K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

template <int TYPE>
cudaError_t launch_logprobs_as(const LogprobArgs& a, cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<TYPE>::Raw);
  const int64_t bytes = a.cols * kEs;
  const int sms = device_sm_count();
  int split = 1;
  while (split < kMaxCluster && a.rows * split < int64_t(sms) * kLpCtas * kStreamWaves &&
         bytes >= split * 2 * kStreamLeast && int64_t(split) * 2 * a.top <= kLpLists)
    split *= 2;
  while (a.rows * split >= (int64_t(1) << 31)) split /= 2;  // CTA numbers are 31 bits
  // batches of a segment, 2^shift of them to a slot
  const int64_t vecs = (a.cols + 2 * (ScoreVec<TYPE>::kCount - 1)) / ScoreVec<TYPE>::kCount;
  const int64_t batches =
      ((vecs + split - 1) / split + Stream<TYPE>::kStep - 1) / Stream<TYPE>::kStep;
  int shift = 0;
  while (((batches - 1) >> shift) >= kLpSlots) ++shift;
  const int slots = static_cast<int>((batches - 1) >> shift) + 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * split));
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = logprobs_smem(a.top, split, slots);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = add_attributes(attr, split);
  auto kern = logprobs_kernel<TYPE>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, kLpMaxSmem, &done);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, kern, a, split, slots, shift);
}

template <int TYPE>
cudaError_t launch_logprobs_backward_as(const LogprobArgs& a, cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<TYPE>::Raw);
  const int64_t bytes = a.cols * kEs;
  const int sms = device_sm_count();
  int split = 1;
  while (split < kMaxCluster && a.rows * split < int64_t(sms) * kLpCtas * kStreamWaves &&
         bytes >= split * 2 * kStreamLeast)
    split *= 2;
  while (a.rows * split >= (int64_t(1) << 31)) split /= 2;
  const bool together = split > 1 && a.grad == a.logits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * split));
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.k + a.top) * 12;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = add_attributes(attr, together ? split : 1);
  auto kern = logprobs_backward_kernel<TYPE>;
  static std::atomic<uint64_t> done{0};
  if (together && split > 8) {
    const cudaError_t e = allow(kern, false, true, &done);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kern, a, split, together);
}

}  // namespace lsdrs
