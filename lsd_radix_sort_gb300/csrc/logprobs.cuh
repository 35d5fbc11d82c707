// K-LOGPROBS: the log probabilities of given tokens, the entropy and the top
// alternatives of rows of logits, and the gradient of all of them.
//
// With y_j = (x_j - m) / t, e_j = exp y_j, S = sum e_j and m the largest score
// of a row:  logp_j = y_j - log S,  H = log S - sum e_j y_j / S.  S and the
// entropy's sum are taken in one pass, both moved along whenever the origin
// of the exponents moves.
#pragma once
#include <algorithm>

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
  const Stats s = moved(v, m, apart2(v.m, origin(m), scale2));
  return {m, warp_sum(s.sum), warp_sum(s.dot)};
}

// A thread's part of it over many vectors; like RunningSoftmax, with the
// products of the exponentials and their exponents as well.
template <int TYPE>
struct RunningStats {
  float o, limit, top, scale, os2;  // exponents are x * scale - os2: see Exponent
  uint64_t sum[2], dot[2];

  __device__ __forceinline__ explicit RunningStats(float scale2)
      : o(-INFINITY), limit(-INFINITY), top(-INFINITY), scale(scale2), os2(0.0f) {
    sum[0] = sum[1] = dot[0] = dot[1] = 0;
  }
  // what the exponents lack because os2 is rounded
  __device__ __forceinline__ float lack() const {
    return o == -INFINITY ? 0.0f : __fmaf_rn(-o, scale, os2);
  }
  __device__ __forceinline__ Stats at_origin() const {
    float a, b, c, d;
    unpack2(add2(sum[0], sum[1]), a, b);
    unpack2(add2(dot[0], dot[1]), c, d);
    const float mend = exp2_approx(lack());
    return {o, (a + b) * mend, (c + d + lack() * (a + b)) * mend};
  }
  __device__ __forceinline__ void move(float m, float scale2) {
    const Stats s = moved(at_origin(), m, apart2(o, m, scale2));
    o = m;
    limit = m + 8.0f / scale2;
    const Exponent e(m, scale2);
    scale = e.scale;
    os2 = e.os2;
    const float a = __fdividef(s.sum, e.mend);
    sum[0] = pack2(a, 0.0f);
    dot[0] = pack2(__fdividef(s.dot, e.mend) - lack() * a, 0.0f);
    sum[1] = dot[1] = 0;
  }
  // Adds vectors, m being their largest score.
  template <int VECS>
  __device__ __forceinline__ void add(const uint4 (&v)[VECS], float m, float scale2) {
    top = fmaxf(top, m);
    if (m > limit) move(m, scale2);
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      uint64_t p[ScoreVec<TYPE>::kCount / 2];
      vec_pairs<TYPE>(v[u], p);
#pragma unroll
      for (int i = 0; i < ScoreVec<TYPE>::kCount / 2; ++i) {
        float a, b;
        unpack2(fma2(p[i], pack2(scale, scale), pack2(-os2, -os2)), a, b);
        const uint64_t y = pack2(above_nothing(a), above_nothing(b));
        const uint64_t x = exp2_2(y);
        sum[i & 1] = add2(sum[i & 1], x);
        dot[i & 1] = fma2(x, y, dot[i & 1]);
      }
    }
  }
  __device__ __forceinline__ Stats result(float scale2) const {
    const Stats s = at_origin();
    return top > o ? moved(s, top, apart2(o, top, scale2)) : s;
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
constexpr uint32_t kOrderMost = 0xFF800000u;   // of +inf; NaN is above

// A score and its column in one word: the larger word is the better score, of
// equal ones the one of the lower column.
__device__ __forceinline__ uint64_t entry_of(uint32_t order, int col) {
  return static_cast<uint64_t>(order) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ uint32_t entry_order(uint64_t e) { return static_cast<uint32_t>(e >> 32); }
__device__ __forceinline__ int entry_col(uint64_t e) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(e));
}

// A call is two kernels.  The first reads the scores once, every warp segments
// of rows of its own, without a pause between two of them, and leaves of each
// segment its statistics and the largest score of every few vectors of a lane
// (a group); it needs that maximum for the softmax anyway.  The second joins
// them, a CTA or a warp per row, and finds the top alternatives: from the groups'
// maxima a bound that `top` of them reach, so that no score below it can be
// among the `top` best, and few others do (of 64 groups about 24 scores reach
// the 20th largest maximum); only groups that reach it are read again.
//
// 4,096 x 131,072 bf16 scores with 20 alternatives take 205 us, of which the
// first kernel has 180 (88% of the measured copy bandwidth) and the second 25,
// bound by latency: three rounds of 9 rows per SM, about 8 us each.  Kernels that
// chose each row's alternatives where its scores were read took 252 us (a CTA
// or a cluster per row) and 254 (one warp of a persistent CTA chooses): the
// loads of other rows then wait for the choice.  Three CTAs per SM: with two
// the first kernel takes 211 us, with four (64 registers) 233.
constexpr int kLpBlock = 256;     // threads of the first kernel's CTAs
constexpr int kLpCtas = 3;        // per SM
constexpr int kLpStep = kWarp * kStreamBatch;  // vectors of a warp's batch
constexpr int kLpSplit = 128;     // segments of a row at most
constexpr int kLpGroups = 4096;   // of a row at most, for lists of up to kLpShort
constexpr int kLpManyGroups = 8192;  // for longer ones
constexpr int kLpFewGroups = 1024;   // that one warp holds
constexpr int kLpShort = 128;     // longest list that is not a long one
constexpr int kLpRadix = 256;

// Candidates held of a row, and groups that may hold them.
__host__ __device__ constexpr inline int candidate_room(int top) {
  return top <= kLpShort ? 512 : 2048;
}
// Shared memory of a selecting CTA: candidates, then groups worth reading again.
__host__ __device__ constexpr inline size_t select_smem(int top) {
  return top == 0 ? 0 : static_cast<size_t>(candidate_room(top)) * 12;
}

// A warp's batch is 2 KB in one piece.  A lane reads every other vector of half
// a 128-byte line, so that its four vectors lie in one line (they are read
// again together) and a load of the warp still takes whole sectors.  (Vectors
// 512 bytes apart: 8,192 x 32,000 bf16 with 20 alternatives 147 us instead of
// 141.  Four neighbouring vectors per lane, by shuffles: 1,368 x 131,072 72 us
// instead of 65.)
__host__ __device__ constexpr inline int lane_vector(int lane) { return lane / 2 * 8 + lane % 2; }
constexpr int kLaneStride = 2;

// How a call's rows are divided: into `split` segments of `per` vectors; a group
// is a lane's vectors of 2^shift batches, or (single) one vector; a segment has
// `slots` of them (a multiple of 8).
struct LpPlan {
  int split, per, shift, slots;
  bool single;
  uint32_t magic;  // 2^32 / slots, rounded up
  __host__ __device__ int groups() const { return split * slots; }
  __device__ __forceinline__ int segment_of(int group) const {
    return static_cast<int>(__umulhi(static_cast<uint32_t>(group), magic));
  }
  // a group's vectors, and the first of them, in its segment
  __device__ __forceinline__ int log_members() const { return single ? 0 : 2 + shift; }
  __device__ __forceinline__ int64_t member(int group, int i) const {
    if (single) return group;
    return ((static_cast<int64_t>(group / kWarp) << shift) + i / kStreamBatch) * kLpStep +
           lane_vector(group % kWarp) + i % kStreamBatch * kLaneStride;
  }
  // the group of a segment's vector
  __device__ __forceinline__ int group_of(int vec) const {
    if (single) return vec;
    return (vec / kLpStep >> shift) * kWarp + vec % kLpStep / 8 * 2 + vec % 2;
  }
};

// Scratch: every segment's statistics, then the groups' maxima (the upper
// halves of their orders; 0 for those that a segment does not reach).
__host__ __device__ inline size_t stats_bytes(int64_t rows, const LpPlan& p) {
  return align_up(static_cast<size_t>(rows) * p.split * sizeof(float4), 256);
}
__device__ __forceinline__ uint16_t* row_groups(const LogprobArgs& a, const LpPlan& p,
                                                int64_t row) {
  return reinterpret_cast<uint16_t*>(static_cast<char*>(a.temp) + stats_bytes(a.rows, p)) +
         row * p.groups();
}

// Segment `rank` of a row: vectors [begin, end).
template <int TYPE>
struct Segment {
  using Raw = typename Score<TYPE>::Raw;
  const Raw* x;
  RowVecs<TYPE> vecs;
  int begin, end;

  __device__ __forceinline__ Segment(const LogprobArgs& a, int64_t row, int rank, int per)
      : x(static_cast<const Raw*>(a.logits) + row * a.stride),
        vecs(x, static_cast<int>(a.cols)) {
    begin = min(rank * per, vecs.count);
    end = min(begin + per, vecs.count);
  }
  __device__ __forceinline__ const uint4* vec0() const {
    return reinterpret_cast<const uint4*>(x - vecs.lead);
  }
};

// What the reading warp needs of a segment from batch to batch; the rest is
// worked out again at a row's ragged ends.
template <int TYPE>
struct Reader {
  const uint4* vec0;
  int begin, end, inner_begin, inner_end;  // inner: whole vectors
  uint32_t item;

  __device__ __forceinline__ Reader(const LogprobArgs& a, uint32_t item_, const LpPlan& p)
      : item(item_) {
    const Segment<TYPE> seg = segment(a, p);
    vec0 = seg.vec0();
    begin = seg.begin;
    end = seg.end;
    inner_begin = seg.vecs.whole_begin();
    inner_end = min(end, seg.vecs.whole_end());
  }
  __device__ __forceinline__ Segment<TYPE> segment(const LogprobArgs& a, const LpPlan& p) const {
    const uint32_t row = item / static_cast<uint32_t>(p.split);
    return Segment<TYPE>(a, row, static_cast<int>(item - row * p.split), p.per);
  }
  __device__ __forceinline__ int batches() const {
    return max(1, (end - begin + kLpStep - 1) / kLpStep);
  }
  // a lane's batch: vectors v0 + u * kLaneStride, -inf past the end
  __device__ __forceinline__ void load(const LogprobArgs& a, const LpPlan& p, int v0,
                                       uint4 (&to)[kStreamBatch]) const {
    constexpr uint32_t kNone = ScoreVec<TYPE>::kMinusInf;
    if (v0 >= inner_begin && v0 + (kStreamBatch - 1) * kLaneStride < inner_end) {
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) to[u] = __ldcs(vec0 + v0 + u * kLaneStride);
    } else {
      const Segment<TYPE> seg = segment(a, p);
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) {
        const int v = v0 + u * kLaneStride;
        to[u] = v < end ? seg.vecs.load(vec0, seg.x, v) : make_uint4(kNone, kNone, kNone, kNone);
      }
    }
  }
};

__device__ __forceinline__ uint32_t upper_order(float x) { return order_of(x) >> 16; }

template <int TYPE>
__device__ __forceinline__ float max_of(const uint4& v) {
  const uint4 one[1] = {v};
  return vec_max<TYPE>(one);
}

// GROUPS: 0 none are kept, 1 of one vector, 4 of a lane's batches.
template <int TYPE, int GROUPS>
__global__ void __launch_bounds__(kLpBlock, kLpCtas)
    logprobs_read_kernel(const __grid_constant__ LogprobArgs a,
                         const __grid_constant__ LpPlan p, const uint32_t items) {
  grid_dependency_sync();
  const uint32_t step = gridDim.x * (kLpBlock / kWarp);
  const uint32_t first = blockIdx.x * (kLpBlock / kWarp) + threadIdx.x / kWarp;
  if (first >= items) return;
  const int lane = static_cast<int>(lane_id()), own = lane_vector(lane);
  auto groups_of = [&](uint32_t item) {  // of a segment
    const uint32_t row = item / static_cast<uint32_t>(p.split);
    return row_groups(a, p, row) + static_cast<int>(item - row * p.split) * p.slots;
  };
  Reader<TYPE> in(a, first, p);
  uint4 r[kStreamBatch], ahead[kStreamBatch];
  in.load(a, p, in.begin + own, r);
  for (uint32_t item = first; item < items; item += step) {
    RunningStats<TYPE> run(a.scale2);
    uint16_t* kept = nullptr;  // this lane's next group
    if (GROUPS != 0) kept = groups_of(item) + (GROUPS == 1 ? own : lane);
    const int batches = in.batches();
    int v = in.begin + own;
    float m = -INFINITY;
    for (int b = 1; b <= batches; ++b) {
      v += kLpStep;
      if (b < batches) {
        in.load(a, p, v, ahead);
      } else if (item + step < items) {  // the next segment's first
        in = Reader<TYPE>(a, item + step, p);
        in.load(a, p, in.begin + own, ahead);
      }
      const float top = vec_max<TYPE>(r);
      if (GROUPS == 1) {
#pragma unroll
        for (int u = 0; u < kStreamBatch; ++u)
          kept[u * kLaneStride] = static_cast<uint16_t>(upper_order(max_of<TYPE>(r[u])));
        kept += kLpStep;
      } else if (GROUPS != 0) {
        m = fmaxf(m, top);
        if ((b & ((1 << p.shift) - 1)) == 0 || b == batches) {
          *kept = static_cast<uint16_t>(upper_order(m));
          kept += kWarp;
          m = -INFINITY;
        }
      }
      run.add(r, top, a.scale2);
#pragma unroll
      for (int u = 0; u < kStreamBatch; ++u) r[u] = ahead[u];
    }
    if (GROUPS != 0) {  // groups that the segment does not reach
      uint16_t* all = groups_of(item);
      const int done =
          GROUPS == 1 ? batches * kLpStep : (((batches - 1) >> p.shift) + 1) * kWarp;
      for (int i = done + lane; i < p.slots; i += kWarp) all[i] = 0;
    }
    const Stats st = warp_join(run.result(a.scale2), a.scale2);
    if (lane == 0)
      static_cast<float4*>(a.temp)[item] = make_float4(st.m, st.sum, st.dot, 0.0f);
  }
}

// Adds to a histogram; lanes with the same digit at once.
__device__ __forceinline__ void count_digit(uint32_t* hist, uint32_t digit) {
  const unsigned active = __activemask();
  const unsigned same = __match_any_sync(active, digit);
  if (lane_id() == static_cast<uint32_t>(__ffs(static_cast<int>(same)) - 1))
    atomicAdd(&hist[digit], static_cast<uint32_t>(__popc(same)));
}

// From the counts of 256 digits: the largest one that `above` plus the counts
// from it on reach `want`, or 0.  `above` becomes the number of those beyond
// it, `reach` that with its own.
__device__ __forceinline__ int pick_digit(const uint32_t* hist, int want, int& above, int& reach) {
  const int lane = static_cast<int>(lane_id());
  // lane 31 has the largest eight digits
  int n[8], mine = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    mine += static_cast<int>(hist[lane * 8 + i]);
    n[i] = mine;  // of this lane's digits, from i on
  }
  int beyond = mine;
#pragma unroll
  for (int o = 1; o < kWarp; o *= 2) {
    const int v = __shfl_down_sync(kFull, beyond, o);
    if (lane + o < kWarp) beyond += v;
  }
  beyond += above - mine;  // above, and of the lanes behind
  const unsigned ok = __ballot_sync(kFull, beyond + mine >= want);
  const int from = ok != 0 ? 31 - __clz(static_cast<int>(ok)) : 0;
  int digit = 0, upto = beyond + mine;
#pragma unroll
  for (int i = 7; i > 0; --i) {
    if (beyond + n[i] >= want) {
      digit = i;
      upto = beyond + n[i];
      break;
    }
  }
  const int over = upto - static_cast<int>(hist[lane * 8 + digit]);
  above = __shfl_sync(kFull, over, from);
  reach = __shfl_sync(kFull, upto, from);
  return __shfl_sync(kFull, lane * 8 + digit, from);
}

// The `top`-th largest of N values of 16 bits per lane, or 0 if that many are
// not above it: bit by bit from the first that they differ in.
template <int N>
__device__ __forceinline__ uint32_t largest_of(const uint32_t (&v)[N], int top) {
  uint32_t all = v[0], any = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    all &= v[i];
    any |= v[i];
  }
  all = __reduce_and_sync(kFull, all);
  any = __reduce_or_sync(kFull, any);
  const int bits = 32 - __clz(static_cast<int>(all ^ any));
  uint32_t best = all >> bits << bits;  // (shared by all of them)
#pragma unroll 1
  for (uint32_t bit = 1u << bits >> 1; bit != 0; bit >>= 1) {
    const uint32_t t = best | bit;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popc(__ballot_sync(kFull, v[i] >= t));
    if (n >= top) best = t;
  }
  return best;
}

// ------------------------------------------------------------- a row, by a CTA
struct RowSelected {
  int hits, count;
  uint32_t words[4][4][kWarp];   // maxima by word, warp, lane
  uint32_t least;
  uint32_t hist[kLpRadix];
  uint64_t prefix;
  int above, reach;
  int part[4];
};

template <int WARPS>
__device__ __forceinline__ void row_sync() {
  if (WARPS == 1)
    __syncwarp();
  else
    __syncthreads();
}

template <int TYPE, int WARPS>
struct Selection {
  static constexpr int kThreads = WARPS * kWarp;
  const LogprobArgs& a;
  const LpPlan& p;
  int64_t row;
  const uint16_t* kept;
  int room;
  uint64_t* cand;
  uint32_t* work;         // groups
  RowSelected* sh;

  // A bound (the upper half of an order) that `top` scores reach, or 0: the
  // `top`-th largest of 64 * WORDS maxima, of this thread's in g.  The first warp
  // finds it for all of them.
  template <int WORDS>
  __device__ __forceinline__ uint32_t bound_of(const uint32_t (&g)[4]) const {
    const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x) / kWarp;
    uint32_t w[WORDS], v[2 * WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = g[i];
#pragma unroll
    for (int i = WORDS; i < 4; ++i) w[i % WORDS] = __vmaxu2(w[i % WORDS], g[i]);
    if constexpr (WARPS > 1) {
      if (warp != 0) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) sh->words[i][warp][lane] = w[i];
      }
      __syncthreads();
    }
    if (warp == 0) {
      if constexpr (WARPS > 1) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
#pragma unroll
          for (int j = 1; j < WARPS; ++j) w[i] = __vmaxu2(w[i], sh->words[i][j][lane]);
      }
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        v[2 * i] = w[i] & 0xFFFFu;
        v[2 * i + 1] = w[i] >> 16;
      }
      const uint32_t best = largest_of(v, a.top);
      if constexpr (WARPS == 1) return best;
      if (lane == 0) sh->least = best;
    }
    if constexpr (WARPS > 1) __syncthreads();
    return sh->least;
  }

  // One digit of a selection by counts: sh->prefix, above, reach.
  __device__ __forceinline__ void pick(uint64_t prefix, int shift, int above) const {
    row_sync<WARPS>();
    if (threadIdx.x < kWarp) {
      int reach;
      const int d = pick_digit(sh->hist, a.top, above, reach);
      if (threadIdx.x == 0) {
        sh->prefix = prefix | static_cast<uint64_t>(d) << shift;
        sh->above = above;
        sh->reach = reach;
      }
    }
    row_sync<WARPS>();
  }
  __device__ __forceinline__ void clear_counts() const {
    for (int i = static_cast<int>(threadIdx.x); i < kLpRadix; i += kThreads) sh->hist[i] = 0;
    row_sync<WARPS>();
  }

  // For long lists every group counts: the digits of their maxima.
  __device__ __forceinline__ uint32_t bound_of_all() const {
    uint64_t prefix = 0;
    int above = 0;
    const int groups = p.groups();
    for (int shift = 8; shift >= 0; shift -= 8) {
      clear_counts();
#pragma unroll 4
      for (int i = static_cast<int>(threadIdx.x); i < groups; i += kThreads) {
        const uint32_t k = kept[i];
        if (shift == 8 || k >> 8 == prefix >> 8) count_digit(sh->hist, k >> shift & 0xFFu);
      }
      pick(prefix, shift, above);
      prefix = sh->prefix;
      above = sh->above;
    }
    return sh->reach < a.top ? 0 : static_cast<uint32_t>(prefix);
  }

  __device__ __forceinline__ void hit(int group) const {
    const int at = atomicAdd(&sh->hits, 1);
    if (at < room) work[at] = static_cast<uint32_t>(group);
  }
  // Lists those of a thread's groups (8 of each vector) that reach the bound.
  template <int VECS>
  __device__ __forceinline__ void hits_of(const uint4 (&v)[VECS], uint32_t largest,
                                          uint32_t least) const {
    const uint32_t below = (least - 1) * 0x10001u;  // (least is not 0)
    if (__vmaxu2(largest, below) == below) return;
    uint32_t reach = 0;  // a bit per group
    static_assert(VECS <= 4);
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const uint32_t words[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t over = __vmaxu2(words[j], below) ^ below;
        if (over & 0xFFFFu) reach |= 1u << (8 * i + 2 * j);
        if (over >> 16) reach |= 2u << (8 * i + 2 * j);
      }
    }
    for (; reach != 0; reach &= reach - 1) {
      const int bit = __ffs(static_cast<int>(reach)) - 1;
      hit((bit / 8 * kThreads + static_cast<int>(threadIdx.x)) * 8 + bit % 8);
    }
  }

  __device__ __forceinline__ void add(uint64_t e) const {
    const int at = atomicAdd(&sh->count, 1);
    if (at < room) cand[at] = e;
  }

  // Candidates: the scores of the listed groups that reach the bound.
  __device__ __forceinline__ void collect(int hits, uint32_t least) const {
    const int log = p.log_members();
    static_assert(kStreamBatch == 4);
    const float from = score_of(least << 16);
    constexpr int kN = ScoreVec<TYPE>::kCount, kAhead = 2;
    const int64_t units = static_cast<int64_t>(hits) << log;
    const Segment<TYPE> whole(a, row, 0, 0);
    for (int64_t u0 = threadIdx.x; u0 < units; u0 += kAhead * kThreads) {
      uint4 r[kAhead];
      int col[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t u = u0 + i * kThreads;
        constexpr uint32_t kNone = ScoreVec<TYPE>::kMinusInf;
        r[i] = make_uint4(kNone, kNone, kNone, kNone);
        col[i] = 0;
        if (u >= units) continue;
        const int g = static_cast<int>(work[u >> log]), rank = p.segment_of(g);
        const int begin = rank * p.per;
        const int64_t v = begin + p.member(g - rank * p.slots,
                                           static_cast<int>(u) & ((1 << log) - 1));
        if (v >= min(begin + p.per, whole.vecs.count)) continue;
        r[i] = whole.vecs.load(whole.vec0(), whole.x, static_cast<int>(v));
        col[i] = static_cast<int>(v) * kN - whole.vecs.lead;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          using Raw = typename Score<TYPE>::Raw;
          const float x = Score<TYPE>::load(
              static_cast<Raw>(kN == 4 ? w[j & 3] : w[j >> 1] >> (16 * (j & 1))));
          if (x >= from) add(entry_of(order_of(x), col[i] + j));
        }
      }
    }
  }

  // f(order, column) for every score of the row that reaches the bound.  NaN is
  // left out, as the groups' maxima and collect() do: counts of scores hold only
  // over one set of them, and say what fits among the candidates.
  template <class F>
  __device__ __forceinline__ void each(uint32_t least, F&& f) const {
    constexpr int kN = ScoreVec<TYPE>::kCount, kAhead = 4;
    for (int rank = 0; rank < p.split; ++rank) {
      const Segment<TYPE> seg(a, row, rank, p.per);
      for (int64_t v0 = seg.begin + static_cast<int>(threadIdx.x); v0 < seg.end;
           v0 += kAhead * kThreads) {
        uint4 r[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int64_t v = v0 + u * kThreads;
          const int off = static_cast<int>(min(v, static_cast<int64_t>(seg.end) - 1) - seg.begin);
          on[u] = v < seg.end && kept[rank * p.slots + p.group_of(off)] >= least;
          if (on[u]) r[u] = seg.vecs.load(seg.vec0(), seg.x, static_cast<int>(v));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (!on[u]) continue;
          const uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
          const int col = static_cast<int>(v0 + u * kThreads) * kN - seg.vecs.lead;
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            using Raw = typename Score<TYPE>::Raw;
            const uint32_t o = order_of(Score<TYPE>::load(
                static_cast<Raw>(kN == 4 ? w[i & 3] : w[i >> 1] >> (16 * (i & 1)))));
            if (o >> 16 >= least && o <= kOrderMost) f(o, col + i);
          }
        }
      }
    }
  }

  // Candidates: the first `want` columns, from the lowest on, whose score has
  // this order.
  __device__ __forceinline__ void first_of(uint32_t least, uint32_t order, int want) const {
    constexpr int kN = ScoreVec<TYPE>::kCount, kEach = 4;
    static_assert(kN * kEach <= 32);
    const Segment<TYPE> whole(a, row, 0, 0);
    const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
    int taken = 0;
    for (int64_t v0 = 0; v0 < whole.vecs.count && taken < want; v0 += kEach * kThreads) {
      const int64_t first = v0 + tid * kEach;  // neighbouring vectors of each thread
      uint32_t equal = 0;
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        if (first + u >= whole.vecs.count) continue;
        const int v = static_cast<int>(first) + u, rank = v / p.per;
        if (kept[rank * p.slots + p.group_of(v - rank * p.per)] < least) continue;
        const uint4 r = whole.vecs.load(whole.vec0(), whole.x, v);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          using Raw = typename Score<TYPE>::Raw;
          const uint32_t o = order_of(Score<TYPE>::load(
              static_cast<Raw>(kN == 4 ? w[i & 3] : w[i >> 1] >> (16 * (i & 1)))));
          if (o == order) equal |= 1u << (u * kN + i);
        }
      }
      int upto = __popc(equal);
      const int own = upto;
#pragma unroll
      for (int o = 1; o < kWarp; o *= 2) {
        const int n = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += n;
      }
      int before = taken + upto - own;
      if (lane == kWarp - 1) sh->part[tid / kWarp] = upto;
      row_sync<WARPS>();
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        if (i < tid / kWarp) before += sh->part[i];
        taken += sh->part[i];
      }
      for (; equal != 0 && before < want; equal &= equal - 1, ++before)
        add(entry_of(order, static_cast<int>(first) * kN + __ffs(static_cast<int>(equal)) - 1 -
                                whole.vecs.lead));
      row_sync<WARPS>();
    }
  }
};

// More candidates than there is room for (many equal scores, or a long list):
// scores are narrowed down digit by digit, 8 bits of their order from the top,
// by counting those that share the digits so far, until what is at and above
// them fits, or is one score: then the lowest columns that have it are looked
// up from the beginning.  (20 of 1,024 x 65,536 equal bf16 scores: 83 us;
// 1,240 with all 64 bits of score and column narrowed down.)
template <int TYPE, int WARPS>
__device__ __noinline__ void select_exactly(const Selection<TYPE, WARPS>& sel, uint32_t least) {
  // the order's bits below are 0 of positive scores and 1 of negative ones
  constexpr int kLast = TYPE == RS_SCORE_BF16 ? 48 : TYPE == RS_SCORE_F16 ? 40 : 32;
  if (threadIdx.x == 0) sel.sh->count = 0;
  row_sync<WARPS>();
  sel.each(least + 1, [&](uint32_t o, int col) { sel.add(entry_of(o, col)); });
  row_sync<WARPS>();
  uint64_t prefix = 0;  // entries from it on are kept, those of its digits divided further
  int shift = 64, above = sel.sh->count;
  // `top` scores reach the bound, so that the last of them has its digits where
  // fewer are beyond it
  const bool known = above < sel.a.top;
  if (known) {
    prefix = static_cast<uint64_t>(least) << 48;
    shift = 48;
  } else {
    above = 0;
  }
  bool more = true;
  while (more && shift > kLast) {
    shift -= 8;
    sel.clear_counts();
    sel.each(least, [&](uint32_t o, int) {
      const uint64_t e = static_cast<uint64_t>(o) << 32;
      if (shift == 56 || (e ^ prefix) >> (shift + 8) == 0)
        count_digit(sel.sh->hist, static_cast<uint32_t>(e >> shift) & 0xFFu);
    });
    sel.pick(prefix, shift, above);
    prefix = sel.sh->prefix;
    above = sel.sh->above;
    more = sel.sh->reach > sel.room;
  }
  const uint32_t order = static_cast<uint32_t>(prefix >> 32) |
                         (prefix >> 63 ? 0u : static_cast<uint32_t>((uint64_t(1) << (kLast - 32)) - 1));
  if (!known || shift != 48) {  // (else those above are there)
    row_sync<WARPS>();
    if (threadIdx.x == 0) sel.sh->count = 0;
    row_sync<WARPS>();
    sel.each(least, [&](uint32_t o, int col) {
      const uint64_t e = entry_of(o, col);
      if (more ? o > order : e >= prefix) sel.add(e);
    });
  }
  if (more) sel.first_of(least, order, sel.a.top - above);
  row_sync<WARPS>();
}

// The same among n candidates in shared memory, until no more than `limit` are
// left.  Worth it for more than twice as many (the 300 best of 16,384 x 2,000
// bf16: 672 us, 1,434 with all 2,000 put in order); for fewer the order costs
// less (128 best of 8,192 x 32,000: 248 us, 311).
template <int TYPE, int WARPS>
__device__ __noinline__ void narrow(const Selection<TYPE, WARPS>& sel, int n, int limit) {
  constexpr int kThreads = WARPS * kWarp;
  const int tid = static_cast<int>(threadIdx.x);
  uint64_t prefix = 0;
  int shift = 64, above = 0;
  do {
    shift -= 8;
    sel.clear_counts();
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t e = sel.cand[i];
      if (shift == 56 || (e ^ prefix) >> (shift + 8) == 0)
        count_digit(sel.sh->hist, static_cast<uint32_t>(e >> shift) & 0xFFu);
    }
    sel.pick(prefix, shift, above);
    prefix = sel.sh->prefix;
    above = sel.sh->above;
  } while (sel.sh->reach > limit && shift > 0);
  if (tid == 0) sel.sh->count = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const uint64_t e = i0 + tid < n ? sel.cand[i0 + tid] : 0;
    row_sync<WARPS>();  // written below are places that have all been read
    if (e >= prefix && e != 0) sel.add(e);
  }
  row_sync<WARPS>();
}

// Puts n entries in order: place(position, entry), the largest first.  There
// is room for the next power of two.
template <int WARPS, class F>
__device__ __forceinline__ void in_order(uint64_t* e, int n, F&& place) {
  constexpr int kThreads = WARPS * kWarp;
  const int tid = static_cast<int>(threadIdx.x);
  if (n <= kThreads) {  // positions are counted
    if (tid < n) {
      const uint64_t own = e[tid];
      int better = 0;
#pragma unroll 4
      for (int i = 0; i < n; ++i) better += e[i] > own;
      place(better, own);
    }
    return;
  }
  if (n <= 4 * kThreads) {
    uint64_t own[4];
    int better[4] = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 4; ++u) own[u] = u * kThreads + tid < n ? e[u * kThreads + tid] : 0;
    for (int i = 0; i < n; ++i) {
      const uint64_t x = e[i];
#pragma unroll
      for (int u = 0; u < 4; ++u) better[u] += x > own[u];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (own[u] != 0) place(better[u], own[u]);
    return;
  }
  int size = 4 * kThreads;
  while (size < n) size *= 2;
  for (int i = n + tid; i < size; i += kThreads) e[i] = 0;
  row_sync<WARPS>();
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      for (int q = tid; q < size / 2; q += kThreads) {
        const int i = (q & ~(step - 1)) * 2 + (q & (step - 1)), j = i + step;
        const uint64_t x = e[i], y = e[j];
        if ((x < y) == ((i & run) == 0)) {
          e[i] = y;
          e[j] = x;
        }
      }
      row_sync<WARPS>();
    }
  for (int i = tid; i < n; i += kThreads) place(i, e[i]);
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
  if (at >= a.top) return;
  a.top_logprobs[row * a.top + at] =
      s.nan ? NAN : s.logprob(score_of(entry_order(e)), a.tau);
  a.top_ids[row * a.top + at] = s.nan ? -1 : entry_col(e);
}

// A thread's first token of a row, asked for before it is needed.
template <int TYPE>
struct Token {
  float x;
  bool live;

  __device__ __forceinline__ Token(const LogprobArgs& a, int64_t row, int k) : x(0.0f), live(false) {
    if (k >= a.k) return;
    const int64_t i = load_index(a.tokens, a.index_bytes, row * a.token_stride + k);
    live = i >= 0 && i < a.cols;
    if (live)
      x = Score<TYPE>::load(
          static_cast<const typename Score<TYPE>::Raw*>(a.logits)[row * a.stride + i]);
  }
};

// All of a row but its `found` alternatives.
template <int TYPE>
__device__ __forceinline__ void store_row(const LogprobArgs& a, int64_t row, const RowStats& s,
                                          const Token<TYPE>& first, int found) {
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  for (int i = found + tid; i < a.top; i += threads) {  // fewer scores than asked for
    a.top_logprobs[row * a.top + i] = s.nan ? NAN : -INFINITY;
    a.top_ids[row * a.top + i] = -1;
  }
  for (int i = tid; i < a.k; i += threads) {
    const Token<TYPE> t = i == tid ? first : Token<TYPE>(a, row, i);
    a.logprobs[row * a.k + i] = t.live ? s.logprob(t.x, a.tau) : 0.0f;
  }
  if (tid == 0) {
    a.entropy[row] = s.entropy;
    a.lse[row] = s.nan ? NAN : s.empty ? -INFINITY : s.m / a.tau + s.log_sum;
    a.stats[row] = make_float2(s.nan ? NAN : s.m, s.log_sum);
  }
}

// The second kernel.  Short lists: a thread's groups stay in its registers.
template <int TYPE, int WARPS>
__global__ void __launch_bounds__(WARPS* kWarp)
    logprobs_rows_kernel(const __grid_constant__ LogprobArgs a, const __grid_constant__ LpPlan p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ RowSelected sh;
  constexpr int kThreads = WARPS * kWarp;
  constexpr int kVecs = (WARPS == 1 ? kLpFewGroups : kLpGroups) / 8 / kThreads;
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  const int64_t row = blockIdx.x;
  if (tid == 0) sh.hits = sh.count = 0;
  grid_dependency_sync();
  const int top = a.top, room = candidate_room(top), groups = p.groups();
  const bool short_list = top > 0 && top <= kLpShort;
  const uint16_t* kept = row_groups(a, p, row);
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int g = (i * kThreads + tid) * 8;
    v[i] = short_list && g < groups ? *reinterpret_cast<const uint4*>(kept + g)
                                    : make_uint4(0, 0, 0, 0);
  }
  const float4* part = static_cast<const float4*>(a.temp) + row * p.split;
  float4 own = lane < p.split ? part[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
  const Token<TYPE> token(a, row, tid);

  const Selection<TYPE, WARPS> sel{
      a, p, row, kept, room, reinterpret_cast<uint64_t*>(smem),
      reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(room) * 8), &sh};
  uint32_t least = 0;
  if (short_list) {
    uint32_t g[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      g[0] = __vmaxu2(g[0], v[i].x);
      g[1] = __vmaxu2(g[1], v[i].y);
      g[2] = __vmaxu2(g[2], v[i].z);
      g[3] = __vmaxu2(g[3], v[i].w);
    }
    least = top <= 32   ? sel.template bound_of<1>(g)
            : top <= 64 ? sel.template bound_of<2>(g)
                        : sel.template bound_of<4>(g);
    least = max(least, kOrderLeast >> 16);
    if (WARPS == 1) __syncwarp();
    sel.hits_of(v, __vmaxu2(__vmaxu2(g[0], g[1]), __vmaxu2(g[2], g[3])), least);
  } else if (top > 0) {
    least = max(sel.bound_of_all(), kOrderLeast >> 16);
    for (int g = tid; g < groups; g += kThreads)
      if (kept[g] >= least) sel.hit(g);
  }
  if (top > 0) {
    row_sync<WARPS>();
    if (sh.hits <= room) sel.collect(sh.hits, least);
  }
  int found = 0;
  if (top > 0) {
    row_sync<WARPS>();
    const bool fits = sh.hits <= room && sh.count <= room;
    row_sync<WARPS>();
    if (!fits) select_exactly(sel, least);
    found = min(sh.count, room);
    int limit = 4 * kThreads;
    while (limit < top) limit *= 2;
    if (WARPS > 1 && found > 2 * limit) {
      row_sync<WARPS>();
      narrow(sel, found, limit);
      found = min(sh.count, room);
    }
    // warps without a result to write
    if (found <= kThreads && tid - lane >= max(found, max(top - found, a.k))) return;
  }
  Stats st{own.x, own.y, own.z};
  for (int i = kWarp + lane; i < p.split; i += kWarp) {
    own = part[i];
    const float m = fmaxf(st.m, own.x), o = origin(m);
    const Stats x = moved(st, m, apart2(st.m, o, a.scale2));
    const Stats y = moved(Stats{own.x, own.y, own.z}, m, apart2(own.x, o, a.scale2));
    st = Stats{m, x.sum + y.sum, x.dot + y.dot};
  }
  const RowStats s(warp_join(st, a.scale2));
  if (top > 0)
    in_order<WARPS>(sel.cand, found, [&](int i, uint64_t e) { store_top(a, row, i, e, s); });
  store_row<TYPE>(a, row, s, token, found);
}

// -------------------------------------------------------------------- backward
// With s the sum of the upstream gradients of a row's tokens and alternatives,
//
//   t dx_j = q_j (g_lse - s - g_H (log q_j + H)) + sum over entries of column j
//
// that is 2^y_j (c0 + c1 y_j) with y_j the exponent from the row's maximum, in
// units of log 2: two multiply-adds and one exponential per score.  The
// entries' columns are written last.  2,048 x 65,536 bf16 in 84 us, 94% of the
// measured copy bandwidth for reading the scores and writing their gradient:
// HBM bounds it.
constexpr int kLpThreads = kStreamThreads;
constexpr int kLpWarps = kLpThreads / kWarp;
struct Pull {
  float c0, c1;
};
// Entries of a row that are compared in pairs; more are sorted by column (2,048 x
// 65,536 bf16: 128 entries 111 us, 121 in pairs; 2,048 entries 332, 4,400).
constexpr int kLpPairs = 64;
__host__ __device__ constexpr inline size_t entries_smem(int n) {
  size_t size = kLpPairs;
  while (size < static_cast<size_t>(n)) size *= 2;
  return n <= kLpPairs ? static_cast<size_t>(n) * 12
                       : (static_cast<size_t>(n) * 12 + 15) / 16 * 16 + size * 8;
}

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
  auto write = [&](int i, float total) {
    const float y = above_nothing(__fmaf_rn(score[i], e.scale, -e.os2));
    g[col[i]] = S::store(exp2_approx(y) * __fmaf_rn(pull.c1, y, pull.c0) +
                         (empty ? 0.0f : total * a.inv_tau));
  };
  // a column named more than once: its first entry writes, for all of them
  if (n <= kLpPairs) {
    for (int i = tid; i < n; i += kLpThreads) {
      const int c = col[i];
      if (c < 0 || c < first || c >= last) continue;
      bool mine = true;
      float total = 0.0f;
      for (int j = 0; j < n && mine; ++j) {
        if (col[j] != c) continue;
        mine = j >= i;
        total += up[j];
      }
      if (mine) write(i, total);
    }
    return;
  }
  // many: by column, then by place
  uint64_t* key = reinterpret_cast<uint64_t*>(smem + (static_cast<size_t>(n) * 12 + 15) / 16 * 16);
  int size = kLpPairs;
  while (size < n) size *= 2;
  for (int i = tid; i < size; i += kLpThreads) {
    const int c = i < n ? col[i] : -1;
    key[i] = c < 0 || c < first || c >= last
                 ? ~uint64_t(0)
                 : static_cast<uint64_t>(c) << 32 | static_cast<uint32_t>(i);
  }
  __syncthreads();
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      for (int q = tid; q < size / 2; q += kLpThreads) {
        const int i = (q & ~(step - 1)) * 2 + (q & (step - 1)), j = i + step;
        const uint64_t x = key[i], y = key[j];
        if ((x > y) == ((i & run) == 0)) {
          key[i] = y;
          key[j] = x;
        }
      }
      __syncthreads();
    }
  for (int i = tid; i < n; i += kLpThreads) {
    const uint64_t own = key[i];
    if (own == ~uint64_t(0) || (i > 0 && key[i - 1] >> 32 == own >> 32)) continue;
    float total = 0.0f;
    for (int j = i; j < n && key[j] >> 32 == own >> 32; ++j)
      total += up[static_cast<uint32_t>(key[j])];
    write(static_cast<int>(static_cast<uint32_t>(own)), total);
  }
}

// ---------------------------------------------------------------------- launch
// The time of `split` segments to a row is that of as many rounds of all warps
// as they take, each at its share of the measured bandwidth, batch by batch,
// and what a segment's end costs.
template <int TYPE>
LpPlan make_logprobs_plan(int64_t rows, int64_t cols, int top, bool aligned, int64_t sms) {
  constexpr int kN = ScoreVec<TYPE>::kCount;
  const int64_t warps = sms * kLpCtas * (kLpBlock / kWarp);
  // (rows that begin anywhere may have parts of one more)
  const int64_t vecs = (cols + (aligned ? 1 : 2) * (kN - 1)) / kN;
  LpPlan p{1, 0, 0, kWarp, false, 0};
  const double ns_per_batch = 16.0 * kLpStep * static_cast<double>(warps) / 6791.0;
  double best = 1e300;
  for (int split = 1; split <= kLpSplit; ++split) {
    const int64_t per = (vecs + split - 1) / split;
    if (split > 1 && per < kLpStep / 2) break;
    const int64_t rounds = (rows * split + warps - 1) / warps;
    const double ns =
        rounds * (static_cast<double>((per + kLpStep - 1) / kLpStep) * ns_per_batch + 500.0);
    if (ns < best) {
      best = ns;
      p.split = split;
    }
  }
  while (p.split > 1 && rows * p.split >= (int64_t(1) << 31)) --p.split;
  p.per = static_cast<int>((vecs + p.split - 1) / p.split);
  const int64_t batches = (p.per + kLpStep - 1) / kLpStep;
  if (top > 0) {
    // single vectors where there are few, or for a long list too few groups of
    // more: the best of short rows are then bounded by several times `top` maxima
    // (16,384 x 2,000 bf16 with 20 alternatives 68 us, 523 with groups of four;
    // 8,192 x 32,000 with 300 in 1,024 groups of four 440, in single ones 625)
    p.single = top <= kLpShort ? p.split * batches * kLpStep <= kLpFewGroups
                               : p.split * batches * kLpStep <= kLpManyGroups &&
                                     p.split * batches * kWarp < 2 * top;
    const int64_t most = top <= kLpShort ? kLpGroups : kLpManyGroups;
    auto slots = [&] {
      return p.single ? batches * kLpStep : (((batches - 1) >> p.shift) + 1) * kWarp;
    };
    while (p.split * slots() > most) ++p.shift;
    p.slots = static_cast<int>(slots());
  }
  p.magic = static_cast<uint32_t>(((uint64_t(1) << 32) + p.slots - 1) / p.slots);
  return p;
}

// The same as the last of this thread, where the sizes are (the search takes a
// microsecond or two, as much as a launch).
template <int TYPE>
LpPlan logprobs_plan(int64_t rows, int64_t cols, int top, bool aligned) {
  struct Last {
    int64_t rows, cols, sms;
    int top;
    LpPlan plan;
  };
  static thread_local Last last[2] = {{-1, 0, 0, 0, {}}, {-1, 0, 0, 0, {}}};
  const int64_t sms = device_sm_count();
  Last& l = last[aligned];
  if (l.rows != rows || l.cols != cols || l.top != top || l.sms != sms)
    l = Last{rows, cols, sms, top, make_logprobs_plan<TYPE>(rows, cols, top, aligned, sms)};
  return l.plan;
}

template <int TYPE>
size_t logprobs_temp(int64_t rows, int64_t cols, int top) {
  size_t most = 0;  // however the rows begin
  for (const bool aligned : {false, true}) {
    const LpPlan p = logprobs_plan<TYPE>(rows, cols, top, aligned);
    most = std::max(most, stats_bytes(rows, p) +
                              (top == 0 ? 0 : static_cast<size_t>(rows) * p.groups() * 2));
  }
  return most;
}

template <int TYPE>
cudaError_t launch_logprobs_as(const LogprobArgs& a, int* launched, cudaStream_t s) {
  const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                       (a.rows == 1 || a.stride % ScoreVec<TYPE>::kCount == 0);
  const LpPlan p = logprobs_plan<TYPE>(a.rows, a.cols, a.top, aligned);
  constexpr int kEach = kLpBlock / kWarp;
  const uint32_t items = static_cast<uint32_t>(a.rows * p.split);
  const uint32_t ctas = std::min<uint32_t>((items + kEach - 1) / kEach,
                                           static_cast<uint32_t>(device_sm_count() * kLpCtas));
  auto read = a.top == 0     ? logprobs_read_kernel<TYPE, 0>
              : p.single     ? logprobs_read_kernel<TYPE, 1>
                             : logprobs_read_kernel<TYPE, 4>;
  const cudaError_t e = launch_kernel(read, dim3(ctas), dim3(kLpBlock), 0, s, a, p, items);
  if (e != cudaSuccess) return e;
  *launched = 2;
  static_assert(select_smem(1024) + sizeof(RowSelected) <= 48 * 1024);
  // A warp per row where there are rows enough for all SMs and a lane holds 32 of
  // its groups: no barriers.  With 20 alternatives 2,500 x 8,000 bf16 takes 33
  // us (39 with four warps), 1,024 x 8,000 27 (23); with 128 8,192 x 32,000 248
  // (290), 2,500 x 8,000 86 (73).
  const bool one_warp = a.top == 0 || (a.top <= kLpShort && p.groups() <= kLpFewGroups &&
                                       a.rows >= (a.top <= 32 ? 2048 : 4096));
  const dim3 rows(static_cast<unsigned>(a.rows));
  return one_warp ? launch_kernel(logprobs_rows_kernel<TYPE, 1>, rows, dim3(kWarp),
                                  select_smem(a.top), s, a, p)
                  : launch_kernel(logprobs_rows_kernel<TYPE, 4>, rows, dim3(4 * kWarp),
                                  select_smem(a.top), s, a, p);
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
  static_assert(entries_smem(2 * RS_MAX_TOP) <= 48 * 1024 - 512);
  cfg.dynamicSmemBytes = entries_smem((a.grad_logprobs != nullptr ? a.k : 0) +
                                      (a.grad_top != nullptr ? a.top : 0));
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
