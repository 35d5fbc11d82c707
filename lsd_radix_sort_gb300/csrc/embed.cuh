// K-EMBED: rows of a table by token, and their gradient.
//
//   out_i = scale * table[id_i]            (zeros for an id outside the table)
//   grad[v] = scale * sum over i with id_i = v of up_i   (in the order of i)
//
// The gradient's tokens are sorted by id, stably, so that each row of the
// table is written once, by those who add it up, in an order that is always
// the same.
#pragma once
#include <type_traits>

#include "scores.cuh"
#include "vocab.h"

namespace lsdrs {

// VEC consecutive elements of a row in one access of up to 32 bytes (a 16-bit
// row's 32-bit gradient in two): as floats, and rounded back.
template <int TYPE, int VEC>
struct Pack {
  using Raw = typename Score<TYPE>::Raw;
  static constexpr int kBytes = VEC * static_cast<int>(sizeof(Raw));
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ static Pack load(const Raw* p) {
    Pack r;
    if constexpr (kBytes >= 32) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.w[i]), "=r"(r.w[i + 1]), "=r"(r.w[i + 2]), "=r"(r.w[i + 3]),
                       "=r"(r.w[i + 4]), "=r"(r.w[i + 5]), "=r"(r.w[i + 6]), "=r"(r.w[i + 7])
                     : "l"(__cvta_generic_to_global(reinterpret_cast<const uint32_t*>(p) + i)));
    } else if constexpr (kBytes == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        r.w[i] = v.x;
        r.w[i + 1] = v.y;
        r.w[i + 2] = v.z;
        r.w[i + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r.w[0] = v.x;
      r.w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      r.w[0] = *p;
    }
    return r;
  }
  __device__ __forceinline__ void store(Raw* p) const {
    if constexpr (kBytes >= 32) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                         __cvta_generic_to_global(reinterpret_cast<uint32_t*>(p) + i)),
                     "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                     "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                     : "memory");
    } else if constexpr (kBytes == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *p = static_cast<Raw>(w[0]);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(Raw) == 4)
      return Score<TYPE>::load(w[i]);
    else
      return Score<TYPE>::load(static_cast<Raw>(w[i / 2] >> (16 * (i & 1))));
  }
  __device__ __forceinline__ static Pack of(const float (&v)[VEC]) {
    Pack r;
    if constexpr (sizeof(Raw) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) r.w[i] = Score<TYPE>::store(v[i]);
    } else if constexpr (VEC == 1) {
      r.w[0] = Score<TYPE>::store(v[0]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2)
        r.w[i / 2] = static_cast<uint32_t>(Score<TYPE>::store(v[i])) |
                     static_cast<uint32_t>(Score<TYPE>::store(v[i + 1])) << 16;
    }
    return r;
  }
  __device__ __forceinline__ static Pack zero() {
    Pack r;
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = 0;
    return r;
  }
};

// A lane's part of a row: VEC consecutive elements, or, of rows that allow only
// UNIT elements (up to 4 bytes) at a time, VEC / UNIT of those, 32 units apart, so
// that a warp's access is still in one piece.  (With one unit per lane, 16,384
// tokens of 2,047 bf16: lookup 94 us, now 31; gradient's rows 130, now 57.)  `left`: elements from the first
// one on to the row's end, at least one (units beyond it are read as the first).
template <int TYPE, int VEC, int UNIT>
struct Part {
  using Unit = Pack<TYPE, UNIT>;
  using Raw = typename Unit::Raw;
  static constexpr int kUnits = VEC / UNIT, kStep = kWarp * UNIT;
  Unit u[kUnits];

  __device__ __forceinline__ static Part load(const Raw* p, int left) {
    Part r;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) r.u[i] = Unit::load(p + (i * kStep < left ? i * kStep : 0));
    return r;
  }
  __device__ __forceinline__ static Part zero() {
    Part r;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) r.u[i] = Unit::zero();
    return r;
  }
  __device__ __forceinline__ void store(Raw* p, int left) const {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (i * kStep < left) u[i].store(p + i * kStep);
  }
  __device__ __forceinline__ float get(int i) const { return u[i / UNIT].get(i % UNIT); }
  // elements 2 * i and 2 * i + 1
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (UNIT > 1 && sizeof(Raw) == 2)
      return ScoreVec<TYPE>::pair(u[2 * i / UNIT].w[i % (UNIT / 2)]);
    else
      return pack2(get(2 * i), get(2 * i + 1));
  }
  __device__ __forceinline__ static Part of(const float (&v)[VEC]) {
    Part r;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      float w[UNIT];
#pragma unroll
      for (int j = 0; j < UNIT; ++j) w[j] = v[i * UNIT + j];
      r.u[i] = Unit::of(w);
    }
    return r;
  }
};
constexpr int kNarrow = 8;  // elements of a lane in narrow accesses

// ---------------------------------------------------------------------- lookup
// One vector per thread and step, two steps at once, over all of the output in
// its order: an id, its row's vector, a store.  Bound by HBM: 65,536 tokens of
// a table of 131,072 x 2,048 bf16 (their ids as frequent as words) in 60 us, 88%
// of the measured copy bandwidth.  With 16-byte vectors 32,768 x 4,096 took 78
// us instead of 72, and with four steps of 32 bytes 72, two 66, one 70.
constexpr int kEmbedThreads = 256;
constexpr int kEmbedBatch = 2;

template <int TYPE, int VEC>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_kernel(const __grid_constant__ EmbedArgs a, const uint32_t per_row) {
  using P = Pack<TYPE, VEC>;
  using Raw = typename P::Raw;
  grid_dependency_sync();
  const Raw* table = static_cast<const Raw*>(a.table);
  Raw* out = static_cast<Raw*>(a.out);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kEmbedThreads * kEmbedBatch);
  const int64_t row0 = base / per_row;
  const uint32_t col0 = static_cast<uint32_t>(base - row0 * per_row);
  int64_t row[kEmbedBatch], id[kEmbedBatch];
  uint32_t col[kEmbedBatch];
#pragma unroll
  for (int u = 0; u < kEmbedBatch; ++u) {
    const uint32_t at = col0 + threadIdx.x + u * kEmbedThreads, down = at / per_row;
    row[u] = row0 + down;
    col[u] = (at - down * per_row) * VEC;
    id[u] = row[u] < a.tokens ? load_index(a.ids, a.index_bytes, row[u]) : -1;
  }
  P p[kEmbedBatch];
#pragma unroll
  for (int u = 0; u < kEmbedBatch; ++u)
    p[u] = id[u] >= 0 && id[u] < a.vocab ? P::load(table + id[u] * a.table_stride + col[u])
                                         : P::zero();
#pragma unroll
  for (int u = 0; u < kEmbedBatch; ++u) {
    if (row[u] >= a.tokens) continue;
    if (a.scale != 1.0f) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = p[u].get(i) * a.scale;
      p[u] = P::of(v);
    }
    // an id outside the table gives zeros, whatever the scale
    if (id[u] < 0 || id[u] >= a.vocab) p[u] = P::zero();
    p[u].store(out + row[u] * a.out_stride + col[u]);
  }
}

// Rows that allow only narrow accesses: a warp per token and 32 * kNarrow columns,
// whose accesses are then in one piece, with one division for all of them.
template <int TYPE, int UNIT>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_narrow_kernel(const __grid_constant__ EmbedArgs a, const uint32_t blocks) {
  using P = Part<TYPE, kNarrow, UNIT>;
  using Raw = typename P::Raw;
  grid_dependency_sync();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kEmbedThreads / kWarp) + threadIdx.x / kWarp;
  const int64_t row = w / blocks;
  const int64_t col = (w - row * blocks) * (kWarp * kNarrow) + lane_id() * UNIT;
  if (row >= a.tokens || col >= a.width) return;
  const int64_t id = load_index(a.ids, a.index_bytes, row);
  const int left = static_cast<int>(a.width - col);
  Raw* out = static_cast<Raw*>(a.out) + row * a.out_stride + col;
  P p = P::zero();  // an id outside the table gives zeros, whatever the scale
  if (id >= 0 && id < a.vocab) {
    p = P::load(static_cast<const Raw*>(a.table) + id * a.table_stride + col, left);
    if (a.scale != 1.0f) {
      float v[kNarrow];
#pragma unroll
      for (int i = 0; i < kNarrow; ++i) v[i] = p.get(i) * a.scale;
      p = P::of(v);
    }
  }
  p.store(out, left);
}

// -------------------------------------------------------------------- gradient
// A token of the sorted list: its place in the call, the row of the output
// that its run of equal ids goes to, and that run's part of the list.
struct __align__(16) Entry {
  uint32_t pos, row, start, end;
};

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / kWarp;
// Rows of a warp under way: with many tokens 4 (rows of 32,768 x 4,096 bf16 96 us
// with their list and cold caches, 113 with 8; three CTAs per SM where accesses are
// of 32 bytes or narrow, four of 16 bytes), with few, where warps are few too, 8.
constexpr int kGradBatch = 4;
constexpr int kFewBatch = 8;

// A thread's sum of VEC columns, two to a register pair.
template <int VEC>
struct Sum {
  static constexpr int kPairs = VEC / 2;
  uint64_t v[kPairs];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = 0;
  }
  template <int TYPE, int UNIT>
  __device__ __forceinline__ void add(const Part<TYPE, VEC, UNIT>& p) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = add2(v[i], p.pair(i));
  }
  __device__ __forceinline__ void add(const Sum& s) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = add2(v[i], s.v[i]);
  }
};

template <int OUT, int VEC, int UNIT>
__device__ __forceinline__ void store_sum(const EmbedGradArgs& a, uint32_t row, int64_t col,
                                          const Sum<VEC>& sum) {
  using O = Part<OUT, VEC, UNIT>;
  typename O::Raw* to = static_cast<typename O::Raw*>(a.out) + row * a.out_stride + col;
  const int left = static_cast<int>(a.width - col);
  float v[VEC];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    unpack2(mul2(sum.v[i], pack2(a.scale, a.scale)), v[2 * i], v[2 * i + 1]);
  if (a.mode == kEmbedAdd) {
    const O was = O::load(to, left);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] += was.get(i);
  }
  O::of(v).store(to, left);
}

// ---- many tokens: the list in memory
// Work is dealt out in chunks of 8 to 32 sorted tokens, a warp for each 32
// vectors of columns.  A warp adds up the
// runs that begin in its chunk, to their ends.  Runs of more than kPiece tokens
// are divided into such pieces, whose sums, in 32 bits, meet in scratch: of
// each 16 neighbours whoever finishes last adds them up, in their order, and
// brings the result to its 16 neighbours.  So a run of any length takes few
// steps one after another (of 32 tokens each; with pieces of 64 that one warp
// added up, the most frequent of 8,191 tokens alone took 30 us; 200,000 tokens
// of one id take 105 us, 1,143 that way).
//
// The gradient of 32,768 x 4,096 bf16 rows takes 70 us after its list, 78% of
// the measured copy bandwidth for the rows read and written: a run's rows lie
// anywhere, and its end waits for its last.  A ring of loads that runs through
// the runs' ends took longer (102 us instead of 93 with the list).  Rows of the
// whole table that no token names are zeroed by CTAs of the same launch, behind
// those that add up: 16,384 tokens into 131,072 x 2,048 bf16 in 100 us, 89% of
// the bandwidth; zeroed beside the list's making they took 111 instead of 105.
constexpr int kMostChunk = 32, kLeastChunk = 8;
constexpr int kPiece = 32;
static_assert(kPiece >= kMostChunk, "a chunk holds the beginnings of two pieces at most");
constexpr int kFan = 16;
constexpr int kLeastBlock = 4 * kWarp;  // columns of a warp at least

// Scratch has two places for each kPiece sorted tokens: two later pieces of
// runs, or two first ones, never begin in the same kPiece (a run with pieces
// is longer than that), a later and a first one may.
__host__ __device__ constexpr inline int64_t piece_places(int64_t tokens) {
  return 2 * ((tokens + kPiece - 1) / kPiece);
}

constexpr int kRunsCount = 0, kRunsLive = 1, kRunsFailed = 2;  // words of the header
struct GradPlan {
  uint32_t* header;
  Entry* list;
  uint32_t* key;         // the id of each run
  float* partial;        // [piece_places][padded width]: later pieces, first pieces
  uint32_t* arrived;     // [piece_places][blocks]: neighbours of the piece there
  int chunk, chunks, blocks;
  int64_t rows_per_zero;
  // where the list is made by the sort of whole keys
  const uint32_t* sort_error;
  uint32_t *keys, *vals, *sorted_keys, *sorted_vals, *slot, *start, *tile_heads;
};

// Brings the sum of a piece to the others of its run.  True for whoever comes
// last of all: `sum` is then that of the run.  A group of neighbours has its
// sum where the first of them had its own, and its counter, at step n, at the
// n-th of them (there are that many wherever a step n is needed).
template <int VEC>
__device__ __forceinline__ bool join_pieces(const GradPlan& p, int block, uint32_t start,
                                         uint32_t end, uint32_t at, Sum<VEC>* sum) {
  using S = Sum<VEC>;
  const int lane = static_cast<int>(lane_id());
  auto place = [&](uint32_t piece) {  // of later pieces, and of first ones
    return 2 * static_cast<int64_t>(start / kPiece + piece) + (piece == 0);
  };
  // 32 * VEC floats: a lane's next pair is 32 pairs on
  auto sums = [&](uint32_t piece) {
    return p.partial + (place(piece) * p.blocks + block) * (kWarp * VEC) + lane * 2;
  };
  auto put = [&](uint32_t piece, const S& v) {
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
      float x, y;
      unpack2(v.v[i], x, y);
      __stcg(reinterpret_cast<float2*>(sums(piece)) + i * kWarp, make_float2(x, y));
    }
  };
  auto get = [&](uint32_t piece) {
    S v;
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
      const float2 f = __ldcg(reinterpret_cast<const float2*>(sums(piece)) + i * kWarp);
      v.v[i] = pack2(f.x, f.y);
    }
    return v;
  };
  uint32_t units = (end - start + kPiece - 1) / kPiece, unit = (at - start) / kPiece;
  uint32_t pieces = 1;  // of a unit
  S mine = *sum;
  for (uint32_t step = 0; units > 1; ++step) {
    const uint32_t first = unit / kFan * kFan, n = min(units - first, uint32_t(kFan));
    if (n > 1) {
      put(unit * pieces, mine);
      __threadfence();
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0)
        before = atomicAdd(&p.arrived[place(first * pieces + step) * p.blocks + block], 1u);
      if (__shfl_sync(kFull, before, 0) != n - 1) return false;
      __threadfence();
      mine.clear();
      constexpr int kAhead = VEC >= 16 ? 2 : VEC >= 8 ? 4 : 8;
      for (uint32_t u0 = 0; u0 < n; u0 += kAhead) {
        S part[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) part[u] = get((first + min(u0 + u, n - 1)) * pieces);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (u0 + u < n) mine.add(part[u]);
      }
    }
    unit = first / kFan;
    units = (units + kFan - 1) / kFan;
    pieces *= kFan;
  }
  *sum = mine;
  return true;
}

template <int IN, int OUT, int VEC, int UNIT>
__device__ __forceinline__ void sum_chunk(const EmbedGradArgs& a, const GradPlan& p, int chunk,
                                          int block) {
  using P = Part<IN, VEC, UNIT>;
  using Raw = typename P::Raw;
  const int lane = static_cast<int>(lane_id());
  const uint32_t live = p.header[kRunsLive];
  const int64_t col = static_cast<int64_t>(block) * kWarp * VEC + lane * UNIT;
  const bool mine = col < a.width;
  const int cols = static_cast<int>(a.width - col);
  const Raw* from = static_cast<const Raw*>(a.grad) + (mine ? col : 0);
  const uint32_t begin = static_cast<uint32_t>(chunk) * p.chunk;
  const Entry none{0, 0, 0, 0};
  Entry e = begin + lane < live ? p.list[begin + lane] : none;
  // A small chunk's rows are all brought to L2 at once, whole 16 bytes of them:
  // the loads below wait for four at a time.  (32,768 rows of 4,096 bf16 94 us,
  // 98 without; 16,384 of 2,047 57, 72.)
  if (p.chunk < kMostChunk && lane < p.chunk && begin + lane < live) {
    const int64_t from_col = static_cast<int64_t>(block) * kWarp * VEC;
    const int64_t n = min(a.width - from_col, static_cast<int64_t>(kWarp * VEC));
    const uint64_t first = static_cast<uint64_t>(__cvta_generic_to_global(
        static_cast<const Raw*>(a.grad) + e.pos * a.grad_stride + from_col));
    const uint64_t low = (first + 15) / 16 * 16, high = (first + n * sizeof(Raw)) / 16 * 16;
    if (low < high)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(low),
                   "r"(static_cast<uint32_t>(high - low))
                   : "memory");
  }
  // where a short run of the chunk may go on
  const Entry next = begin + kWarp + lane < live ? p.list[begin + kWarp + lane] : none;
  const unsigned pieces = __ballot_sync(kFull, lane < p.chunk && begin + lane < live &&
                                                   e.end - e.start > kPiece &&
                                                   (begin + lane - e.start) % kPiece == 0);
  const uint32_t long_start = e.start, long_end = e.end;
  Sum<VEC> sum;
  sum.clear();
#pragma unroll 1
  for (int window = 0; window < 2; ++window) {  // short runs that begin in the chunk
    const uint32_t at = begin + window * kWarp + lane;
    if (window == 1) e = next;
    const bool ours = at < live && e.end - e.start <= kPiece && e.start >= begin &&
                      e.start < begin + p.chunk;
    const unsigned ends = __ballot_sync(kFull, at + 1 == e.end);
    unsigned todo = __ballot_sync(kFull, ours);
    while (todo != 0) {
      P r[kGradBatch];
      unsigned left = todo;
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        const uint32_t pos = __shfl_sync(kFull, e.pos, __ffs(static_cast<int>(left)) - 1);
        r[u] = mine && left != 0 ? P::load(from + pos * a.grad_stride, cols) : P::zero();
        left &= left - 1;
      }
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        if (todo != 0) {
          const int t = __ffs(static_cast<int>(todo)) - 1;
          todo &= todo - 1;
          sum.add(r[u]);
          if ((ends >> t & 1) != 0) {
            const uint32_t row = __shfl_sync(kFull, e.row, t);
            if (mine) store_sum<OUT, VEC, UNIT>(a, row, col, sum);
            sum.clear();
          }
        }
      }
    }
  }
#pragma unroll 1
  for (unsigned todo = pieces; todo != 0; todo &= todo - 1) {  // two at most
    const int t = __ffs(static_cast<int>(todo)) - 1;
    const uint32_t start = __shfl_sync(kFull, long_start, t);
    const uint32_t end = __shfl_sync(kFull, long_end, t), first = begin + t;
    const int n = static_cast<int>(min(end - first, static_cast<uint32_t>(kPiece)));
    const Entry own = lane < n ? p.list[first + lane] : none;
    sum.clear();
    for (int i = 0; i < n; i += kGradBatch) {
      P r[kGradBatch];
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        const uint32_t pos = __shfl_sync(kFull, own.pos, (i + u) % kWarp);
        r[u] = mine && i + u < n ? P::load(from + pos * a.grad_stride, cols) : P::zero();
      }
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u)
        if (i + u < n) sum.add(r[u]);
    }
    const uint32_t row = __shfl_sync(kFull, own.row, 0);
    if (join_pieces<VEC>(p, block, start, end, first, &sum) && mine)
      store_sum<OUT, VEC, UNIT>(a, row, col, sum);
  }
}

// A token's sort key: its id, or the table's length for one without a row.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t i) {
  const int64_t id = load_index(a.ids, a.index_bytes, i);
  return static_cast<uint32_t>(id < 0 || id >= a.vocab || id == a.padding_id ? a.vocab : id);
}

// Zeros (or `fill`) for the rows of the table [first, last) that are not marked.
template <int OUT>
__device__ __forceinline__ void fill_rows(const EmbedGradArgs& a, int64_t first, int64_t last,
                                          float fill, const uint32_t* named) {
  using Raw = typename Score<OUT>::Raw;
  const Raw raw = Score<OUT>::store(fill);
  const uint32_t word = sizeof(Raw) == 4 ? raw : raw | static_cast<uint32_t>(raw) << 16;
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  for (int64_t v = first + tid / kWarp; v < last; v += blockDim.x / kWarp) {
    if (named[(v - first) / 32] >> ((v - first) % 32) & 1) continue;
    Raw* to = static_cast<Raw*>(a.out) + v * a.out_stride;
    // 16 bytes at a time where they are aligned
    const int lead = static_cast<int>((16 - reinterpret_cast<uintptr_t>(to) % 16) % 16 / sizeof(Raw));
    const int64_t head = min(static_cast<int64_t>(lead), a.width);
    constexpr int kN = 16 / static_cast<int>(sizeof(Raw));
    const int64_t vecs = (a.width - head) / kN;
    if (lane < head) to[lane] = raw;
    for (int64_t i = lane; i < vecs; i += kWarp)
      __stcs(reinterpret_cast<uint4*>(to + head) + i, make_uint4(word, word, word, word));
    const int64_t tail = head + vecs * kN + lane;
    if (tail < a.width) to[tail] = raw;
  }
}

// The same of those that no run names; key: the ids of the runs, in order, in
// memory or shared memory.
template <int OUT>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, const uint32_t* key, int runs,
                                          int64_t first, int64_t last, float fill,
                                          uint32_t* named) {
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  const int threads = static_cast<int>(blockDim.x);
  const int words = static_cast<int>((last - first + 31) / 32);
  for (int i = tid; i < words; i += threads) named[i] = 0;
  __syncthreads();
  // the first run of an id >= first: 32 places are looked up at a time
  int lo = 0, hi = runs;  // it is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + kWarp - 1) / kWarp;
    const int at = lo + lane * step;
    const unsigned below = __ballot_sync(kFull, at < hi && static_cast<int64_t>(key[at]) < first);
    const int n = __popc(below);  // places below: a prefix of them
    if (n == 0) break;
    const int left = lo + (n - 1) * step;
    hi = min(hi, left + step);
    lo = left + 1;
  }
  for (int i = lo + tid; i < runs; i += threads) {
    const int64_t v = static_cast<int64_t>(key[i]) - first;
    if (v >= last - first) break;
    atomicOr(&named[v / 32], 1u << (v % 32));
  }
  __syncthreads();
  fill_rows<OUT>(a, first, last, fill, named);
}

constexpr int kZeroMostRows = 4096;  // of one CTA

template <int IN, int OUT, int VEC, int UNIT>
__global__ void __launch_bounds__(
    kGradThreads, VEC * sizeof(typename Score<IN>::Raw) == 32 || UNIT < VEC ? 3 : 4)
    embed_grad_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p,
                      const int64_t sum_ctas) {
  static_assert(kWarp * VEC >= kLeastBlock && kWarp * VEC <= (VEC == 16 ? 512 : 256));
  __shared__ uint32_t named[kZeroMostRows / 32];
  grid_dependency_sync();
  const int64_t cta = blockIdx.x;
  if (cta >= sum_ctas) {
    const int64_t first = (cta - sum_ctas) * p.rows_per_zero;
    zero_rows<OUT>(a, p.key, static_cast<int>(p.header[kRunsCount]), first,
                   min(first + p.rows_per_zero, a.vocab),
                   p.header[kRunsFailed] != 0 ? NAN : 0.0f, named);
    return;
  }
  const int64_t w = cta * kGradWarps + threadIdx.x / kWarp, chunk = w / p.blocks;
  if (chunk < p.chunks)
    sum_chunk<IN, OUT, VEC, UNIT>(a, p, static_cast<int>(chunk), static_cast<int>(w % p.blocks));
}

// ---- few tokens: every CTA makes the list by itself
// Up to kFewTokens: each CTA sorts the tokens' (id, place) in shared memory, all
// alike, which is quicker than telling each other, and takes its part of the
// runs: a warp per run and 32 vectors of columns, all warps of a CTA together
// where a run is longer than kLongRun.  Bound by the latency of the sort's two
// or three digits: 512 x 512 f16 rows take 9 us on the device.  2,048 x 512 bf16
// rows take 14 us, 31 by way of the list in memory; 2,048 x 4,096 27 and 35.
constexpr int kFewTokens = 2048;
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / kWarp;
constexpr int kLongRun = 16;

// Ranks of a warp's 32 * ITEMS words by a digit, in their order: a word's place
// among the warp's of its digit, and how many each digit has.  (By the match
// instruction instead of a ballot per bit the gradient of 2,048 tokens took 49
// us instead of 43, before other steps.)
constexpr int kMaxRadix = 512;
template <int ITEMS, class W>
__device__ __forceinline__ void rank_words(const W (&w)[ITEMS], int shift, int bits,
                                           uint16_t* counts, uint32_t (&place)[ITEMS]) {
  const uint32_t radix = 1u << bits;
  for (uint32_t i = lane_id(); i < radix / 8 + 1 && i < kMaxRadix / 8; i += kWarp)
    reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const uint32_t d = static_cast<uint32_t>(w[u] >> shift) & (radix - 1);
    unsigned same = kFull;
    for (int b = 0; b < bits; ++b) {
      const unsigned set = __ballot_sync(kFull, d >> b & 1);
      same &= (d >> b & 1) != 0 ? set : ~set;
    }
    const unsigned before = same & lanemask_lt();
    const uint32_t was = counts[d];
    __syncwarp();
    place[u] = was + __popc(before);
    if (before == 0) counts[d] = static_cast<uint16_t>(was + __popc(same));
    __syncwarp();
  }
}

// A digit's counts by warp become those of the warps before; returns their sum.
template <int WARPS>
__device__ __forceinline__ uint32_t sum_warps(uint16_t (*counts)[kMaxRadix], uint32_t digit) {
  uint32_t n[WARPS], total = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) n[i] = counts[i][digit];
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    counts[i][digit] = static_cast<uint16_t>(total);
    total += n[i];
  }
  return total;
}

// Sums of v over the threads before this one; all: over all of them.
template <int WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t* all) {
  const uint32_t lane = lane_id(), warp = threadIdx.x / kWarp;
  uint32_t upto = v;
#pragma unroll
  for (int o = 1; o < kWarp; o *= 2) {
    const uint32_t n = __shfl_up_sync(kFull, upto, o);
    if (lane >= static_cast<uint32_t>(o)) upto += n;
  }
  __syncthreads();  // (what was there before has been read)
  if (lane == kWarp - 1) part[warp] = upto;
  __syncthreads();
  const uint32_t n = lane < WARPS ? part[lane] : 0;
  *all = __reduce_add_sync(kFull, n);
  return __reduce_add_sync(kFull, lane < warp ? n : 0) + upto - v;
}

// W: words that hold an id and a place (shift bits), 32 or 64 bits.
template <class W>
struct FewShared {
  uint16_t counts[kFewWarps][kMaxRadix];
  W word[kFewTokens];
  uint32_t base[kMaxRadix];
  uint32_t key[kFewTokens];        // of each run
  uint16_t start[kFewTokens + 8];
  uint16_t long_run[kFewTokens / kLongRun];
  uint32_t part[kWarp];
  uint32_t named[kZeroMostRows / 32];
};

// The tokens in order of their ids, ITEMS per thread.
template <int ITEMS, class W>
__device__ __forceinline__ void sort_few(const EmbedGradArgs& a, FewShared<W>& sh, int shift,
                                         int passes, int bits) {
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int first = warp * kWarp * ITEMS + static_cast<int>(lane_id());
  W w[ITEMS];
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const int i = first + u * kWarp;
    w[u] = i < a.tokens ? static_cast<W>(key_of(a, i)) << shift | static_cast<W>(i)
                        : ~static_cast<W>(0);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int at = shift + pass * bits;
    uint32_t place[ITEMS], all;
    rank_words<ITEMS>(w, at, bits, sh.counts[warp], place);
    __syncthreads();
    const bool digit = tid < 1 << bits;
    const uint32_t total = digit ? sum_warps<kFewWarps>(sh.counts, tid) : 0;
    const uint32_t smaller = block_scan<kFewWarps>(total, sh.part, &all);
    if (digit) sh.base[tid] = smaller;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
      const uint32_t d = static_cast<uint32_t>(w[u] >> at) & ((1u << bits) - 1);
      sh.word[sh.base[d] + sh.counts[warp][d] + place[u]] = w[u];
    }
    __syncthreads();
    if (pass + 1 < passes) {
#pragma unroll
      for (int u = 0; u < ITEMS; ++u) w[u] = sh.word[first + u * kWarp];
    }
  }
}

// The sum of rows [from, to) of the list.
template <int IN, int VEC, int UNIT, class W>
__device__ __forceinline__ Sum<VEC> sum_rows(const EmbedGradArgs& a, const W* word, W places,
                                             int from, int to, int64_t col) {
  using P = Part<IN, VEC, UNIT>;
  const auto* up = static_cast<const typename P::Raw*>(a.grad) + col;
  const int cols = static_cast<int>(a.width - col);
  Sum<VEC> sum;
  sum.clear();
  for (int t = from; t < to; t += kFewBatch) {
    P r[kFewBatch];
#pragma unroll
    for (int u = 0; u < kFewBatch; ++u)
      r[u] = t + u < to
                 ? P::load(up + static_cast<int64_t>(word[t + u] & places) * a.grad_stride, cols)
                 : P::zero();
#pragma unroll
    for (int u = 0; u < kFewBatch; ++u)
      if (t + u < to) sum.add(r[u]);
  }
  return sum;
}

template <int IN, int OUT, int VEC, int UNIT, class W>
__global__ void __launch_bounds__(kFewThreads)
    embed_grad_few_kernel(const __grid_constant__ EmbedGradArgs a, const int shift,
                          const int passes, const int bits, const int blocks, const int sum_ctas,
                          const int64_t rows_per_zero) {
  extern __shared__ __align__(16) unsigned char smem[];
  FewShared<W>& sh = *reinterpret_cast<FewShared<W>*>(smem);
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int lane = static_cast<int>(lane_id());
  grid_dependency_sync();
  constexpr int kEach = kFewTokens / kFewThreads;
  const int tokens = static_cast<int>(a.tokens), cta = static_cast<int>(blockIdx.x);
  if (cta >= sum_ctas) {  // the zeros need no order
    const int64_t first = (cta - sum_ctas) * rows_per_zero;
    const int64_t last = min(first + rows_per_zero, a.vocab);
    for (int i = tid; i < kZeroMostRows / 32; i += kFewThreads) sh.named[i] = 0;
    __syncthreads();
    for (int i = tid; i < tokens; i += kFewThreads) {
      const int64_t v = static_cast<int64_t>(key_of(a, i)) - first;
      if (v >= 0 && v < last - first) atomicOr(&sh.named[v / 32], 1u << (v % 32));
    }
    __syncthreads();
    fill_rows<OUT>(a, first, last, 0.0f, sh.named);
    return;
  }
  const int each = tokens > kFewThreads ? kEach : 1, base = tid * each;
  if (each == 1)
    sort_few<1>(a, sh, shift, passes, bits);
  else
    sort_few<kEach>(a, sh, shift, passes, bits);
  // its runs: the places where a live id differs from the one before
  uint32_t heads = 0, live = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int i = base + u;
    if (u >= each || i >= tokens) break;
    const W key = sh.word[i] >> shift;
    if (key >= static_cast<W>(a.vocab)) break;
    ++live;
    if (i == 0 || sh.word[i - 1] >> shift != key) heads |= 1u << u;
  }
  uint32_t all;  // runs and tokens at once
  int run = static_cast<int>(
      block_scan<kFewWarps>(static_cast<uint32_t>(__popc(heads)) << 16 | live, sh.part, &all) >>
      16);
  const int runs = static_cast<int>(all >> 16);
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    if ((heads >> u & 1) == 0) continue;
    sh.key[run] = static_cast<uint32_t>(sh.word[base + u] >> shift);
    sh.start[run++] = static_cast<uint16_t>(base + u);
  }
  if (tid == 0) sh.start[runs] = static_cast<uint16_t>(all & 0xFFFFu);
  __syncthreads();

  if (a.mode == kEmbedRows && blockIdx.x == 0) {
    const int64_t rows = min(a.tokens, a.vocab);
    for (int i = tid; i < rows; i += kFewThreads)
      a.row_ids[i] = i < runs ? static_cast<int64_t>(sh.key[i]) : -1;
    if (tid == 0) *a.count = runs;
  }
  const W places = (static_cast<W>(1) << shift) - 1;
  const int items = runs * blocks;
  auto row_of = [&](int r) { return a.mode == kEmbedRows ? static_cast<uint32_t>(r) : sh.key[r]; };
  // long runs, in as many parts as warps, joined in their order; every CTA lists
  // them in the same order
  uint32_t longs = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u)
    if (u < each && base + u < runs && sh.start[base + u + 1] - sh.start[base + u] > kLongRun)
      longs |= 1u << u;
  uint32_t long_runs;
  uint32_t nth = block_scan<kFewWarps>(static_cast<uint32_t>(__popc(longs)), sh.part, &long_runs);
#pragma unroll
  for (int u = 0; u < kEach; ++u)
    if ((longs >> u & 1) != 0) sh.long_run[nth++] = static_cast<uint16_t>(base + u);
  __syncthreads();
  uint64_t* parts = reinterpret_cast<uint64_t*>(smem + sizeof(FewShared<W>));
  for (int w = cta; w < static_cast<int>(long_runs) * blocks; w += sum_ctas) {
    const int n = w / blocks, r = sh.long_run[n], from = sh.start[r], to = sh.start[r + 1];
    const int64_t col = static_cast<int64_t>(w - n * blocks) * kWarp * VEC + lane * UNIT;
    const int per = (to - from + kFewWarps - 1) / kFewWarps;
    Sum<VEC> sum;
    if (col < a.width) {
      sum = sum_rows<IN, VEC, UNIT, W>(a, sh.word, places, min(from + warp * per, to),
                                 min(from + (warp + 1) * per, to), col);
#pragma unroll
      for (int i = 0; i < Sum<VEC>::kPairs; ++i)
        parts[(warp * Sum<VEC>::kPairs + i) * kWarp + lane] = sum.v[i];
    }
    __syncthreads();
    if (warp == 0 && col < a.width) {
      for (int n = 1; n < kFewWarps; ++n)
#pragma unroll
        for (int i = 0; i < Sum<VEC>::kPairs; ++i)
          sum.v[i] = add2(sum.v[i], parts[(n * Sum<VEC>::kPairs + i) * kWarp + lane]);
      store_sum<OUT, VEC, UNIT>(a, row_of(r), col, sum);
    }
    __syncthreads();
  }
  for (int w = cta * kFewWarps + warp; w < items; w += sum_ctas * kFewWarps) {
    const int r = w / blocks, from = sh.start[r], to = sh.start[r + 1];
    const int64_t col = static_cast<int64_t>(w - r * blocks) * kWarp * VEC + lane * UNIT;
    if (to - from > kLongRun || col >= a.width) continue;
    store_sum<OUT, VEC, UNIT>(a, row_of(r), col,
                        sum_rows<IN, VEC, UNIT, W>(a, sh.word, places, from, to, col));
  }
}

}  // namespace lsdrs
