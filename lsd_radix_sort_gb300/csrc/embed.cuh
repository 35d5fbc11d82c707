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

// VEC consecutive elements of a row in one access (16 bytes at most per
// instruction): as floats, and rounded back.
template <int TYPE, int VEC>
struct Pack {
  using Raw = typename Score<TYPE>::Raw;
  static constexpr int kBytes = VEC * static_cast<int>(sizeof(Raw));
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ static Pack load(const Raw* p) {
    Pack r;
    if constexpr (kBytes >= 16) {
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
    if constexpr (kBytes >= 16) {
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

// ---------------------------------------------------------------------- lookup
// One vector per thread and step, four steps at once, over all of the output
// in its order: an id, its row's vector, a store.
constexpr int kEmbedThreads = 256;
constexpr int kEmbedBatch = 4;

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

// -------------------------------------------------------------------- gradient
// A token of the sorted list: its place in the call, the row of the output
// that its run of equal ids goes to, and that run's part of the list.
struct __align__(16) Entry {
  uint32_t pos, row, start, end;
};

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / kWarp;
constexpr int kGradBatch = 8;   // rows of a warp under way

template <int IN, int OUT, int VEC>
__device__ __forceinline__ void store_sum(const EmbedGradArgs& a, uint32_t row, int64_t col,
                                          const float (&sum)[VEC]) {
  using O = Pack<OUT, VEC>;
  typename O::Raw* to = static_cast<typename O::Raw*>(a.out) + row * a.out_stride + col;
  float v[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = sum[i] * a.scale;
  if (a.mode == kEmbedAdd) {
    const O was = O::load(to);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] += was.get(i);
  }
  O::of(v).store(to);
}

// ---- many tokens: the list in memory
// Work is dealt out in chunks of kChunk sorted tokens, a warp for each 32
// vectors of columns.  A warp adds up the runs that begin in its chunk, to
// their ends.  Runs of more than kPiece tokens are divided into such pieces,
// whose sums, in 32 bits, meet in scratch: whoever finishes a run's last
// piece adds them up, in their order.
constexpr int kChunk = 32;
constexpr int kPiece = 64;
static_assert(kPiece >= kChunk, "a chunk holds the beginnings of two pieces at most");

constexpr int kRunsCount = 0, kRunsLive = 1, kRunsFailed = 2;  // words of the header
struct GradPlan {
  uint32_t* header;
  Entry* list;
  uint32_t* key;         // the id of each run
  float* partial;        // [2 * chunks][padded width]: later pieces, first pieces
  uint32_t* arrived;     // [chunks][blocks]: pieces of the run that begins there
  int chunks, blocks;
  int64_t rows_per_zero;
  // where the list is made by the sort of whole keys
  const uint32_t* sort_error;
  uint32_t *keys, *vals, *sorted_keys, *sorted_vals, *slot, *start, *tile_heads;
};

template <int VEC>
struct Sum {
  float v[VEC];
};

// The sum of a piece; the last of its run's to arrive gets the whole sum, in
// `sum`, and true.
template <int VEC>
__device__ __noinline__ bool join_pieces(const GradPlan& p, int block, uint32_t start,
                                         uint32_t end, uint32_t at, Sum<VEC>* sum) {
  const int lane = static_cast<int>(lane_id());
  const int64_t padded = static_cast<int64_t>(p.blocks) * kWarp * VEC;
  const int64_t col = (static_cast<int64_t>(block) * kWarp + lane) * VEC;
  const uint32_t pieces = (end - start + kPiece - 1) / kPiece, number = (at - start) / kPiece;
  auto place = [&](uint32_t n) {
    return p.partial + (2 * static_cast<int64_t>((start + n * kPiece) / kChunk) + (n == 0)) * padded +
           col;
  };
#pragma unroll
  for (int i = 0; i < VEC; ++i) __stcg(place(number) + i, sum->v[i]);
  __threadfence();
  __syncwarp();
  uint32_t before = 0;
  if (lane == 0)
    before = atomicAdd(&p.arrived[static_cast<int64_t>(start / kChunk) * p.blocks + block], 1u);
  if (__shfl_sync(kFull, before, 0) != pieces - 1) return false;
  __threadfence();
  Sum<VEC> all;
#pragma unroll
  for (int i = 0; i < VEC; ++i) all.v[i] = 0.0f;
  constexpr int kAhead = VEC >= 8 ? 4 : 8;
  for (uint32_t n0 = 0; n0 < pieces; n0 += kAhead) {
    float v[kAhead][VEC];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const float* from = place(min(n0 + n, pieces - 1));
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[n][i] = __ldcg(from + i);
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n)
      if (n0 + n < pieces)
#pragma unroll
        for (int i = 0; i < VEC; ++i) all.v[i] += v[n][i];
  }
  *sum = all;
  return true;
}

template <int IN, int OUT, int VEC>
__device__ __forceinline__ void sum_chunk(const EmbedGradArgs& a, const GradPlan& p, int chunk,
                                          int block) {
  using P = Pack<IN, VEC>;
  using Raw = typename P::Raw;
  const int lane = static_cast<int>(lane_id());
  const uint32_t live = p.header[kRunsLive];
  const int64_t col = (static_cast<int64_t>(block) * kWarp + lane) * VEC;
  const bool mine = col < a.width;
  const Raw* from = static_cast<const Raw*>(a.grad) + (mine ? col : 0);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  bool open = false;  // a piece is under way
  for (uint32_t window = chunk * kChunk; window < live; window += kChunk) {
    const uint32_t at = window + lane;
    Entry e{0, 0, 0, 0};
    if (at < live) e = p.list[at];
    const unsigned begins = __ballot_sync(kFull, at < live && (at - e.start) % kPiece == 0);
    const unsigned ends = __ballot_sync(
        kFull, at < live && (at + 1 == e.end || (at + 1 - e.start) % kPiece == 0));
    int t = 0, last;  // tokens [t, last) of the window are this warp's
    if (open) {       // what began before, to its end
      last = ends != 0 ? __ffs(static_cast<int>(ends)) : kWarp;
    } else {
      if (begins == 0) return;
      t = __ffs(static_cast<int>(begins)) - 1;
      last = static_cast<int>(min(static_cast<uint32_t>(kWarp), live - window));
    }
#pragma unroll 1
    for (; t < last; t += kGradBatch) {
      P r[kGradBatch];
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        const uint32_t pos = __shfl_sync(kFull, e.pos, min(t + u, kWarp - 1));
        r[u] = mine && t + u < last ? P::load(from + pos * a.grad_stride) : P::zero();
      }
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        if (t + u < last) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) sum[i] += r[u].get(i);
          if ((ends >> (t + u) & 1) != 0) {  // the end of a run, or of a piece of one
            const uint32_t b = __shfl_sync(kFull, e.start, t + u);
            const uint32_t n = __shfl_sync(kFull, e.end, t + u) - b;
            const uint32_t row = __shfl_sync(kFull, e.row, t + u);
            bool whole = true;
            if (n > kPiece) {
              Sum<VEC> s;
#pragma unroll
              for (int i = 0; i < VEC; ++i) s.v[i] = sum[i];
              whole = join_pieces<VEC>(p, block, b, b + n, window + t + u, &s);
#pragma unroll
              for (int i = 0; i < VEC; ++i) sum[i] = s.v[i];
            }
            if (whole && mine) store_sum<IN, OUT, VEC>(a, row, col, sum);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
          }
        }
      }
    }
    open = last == kWarp && (ends >> (kWarp - 1)) == 0;
    if (!open) return;
  }
}

// Zeros (or `fill`) for the rows of the table [first, last) that no run names;
// key: the ids of the runs, in order, in memory or shared memory.
template <int OUT>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, const uint32_t* key, int runs,
                                          int64_t first, int64_t last, float fill,
                                          uint32_t* named) {
  using Raw = typename Score<OUT>::Raw;
  const Raw raw = Score<OUT>::store(fill);
  const uint32_t word = sizeof(Raw) == 4 ? raw : raw | static_cast<uint32_t>(raw) << 16;
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
  for (int64_t v = first + tid / kWarp; v < last; v += threads / kWarp) {
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

constexpr int kZeroMostRows = 4096;  // of one CTA

template <int IN, int OUT, int VEC>
__global__ void __launch_bounds__(kGradThreads, VEC * sizeof(typename Score<IN>::Raw) == 16 ? 3 : 4)
    embed_grad_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p,
                      const int64_t sum_ctas) {
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
    sum_chunk<IN, OUT, VEC>(a, p, static_cast<int>(chunk), static_cast<int>(w % p.blocks));
}

// ---- few tokens: every CTA makes the list by itself
// Up to kFewTokens: each CTA sorts the tokens' (id, place) in shared memory, all
// alike, which is quicker than telling each other, and takes its part of the
// runs: a warp per run and 32 vectors of columns, all warps of a CTA together
// where a run is longer than kLongRun.
constexpr int kFewTokens = 2048;
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / kWarp;
constexpr int kLongRun = 64;

// A token's sort key: its id, or the table's length for one without a row.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t i) {
  const int64_t id = load_index(a.ids, a.index_bytes, i);
  return static_cast<uint32_t>(id < 0 || id >= a.vocab || id == a.padding_id ? a.vocab : id);
}

// W: words that hold an id and a place (shift bits), 32 or 64 bits.
template <class W>
struct FewShared {
  W word[kFewTokens];
  uint32_t key[kFewTokens];        // of each run
  uint16_t start[kFewTokens + 1];
  uint32_t part[kFewWarps];
  uint32_t named[kZeroMostRows / 32];
};

// The sum of rows [from, to) of the list.
template <int IN, int VEC, class W>
__device__ __forceinline__ void sum_rows(const EmbedGradArgs& a, const W* word, W places, int from,
                                         int to, int64_t col, float (&sum)[VEC]) {
  using P = Pack<IN, VEC>;
  const auto* up = static_cast<const typename P::Raw*>(a.grad) + col;
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  for (int t = from; t < to; t += kGradBatch) {
    P r[kGradBatch];
#pragma unroll
    for (int u = 0; u < kGradBatch; ++u)
      r[u] = t + u < to ? P::load(up + static_cast<int64_t>(word[t + u] & places) * a.grad_stride)
                        : P::zero();
#pragma unroll
    for (int u = 0; u < kGradBatch; ++u)
      if (t + u < to)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += r[u].get(i);
  }
}

template <int IN, int OUT, int VEC, class W>
__global__ void __launch_bounds__(kFewThreads)
    embed_grad_few_kernel(const __grid_constant__ EmbedGradArgs a, const int size, const int shift,
                          const int blocks, const int sum_ctas, const int64_t rows_per_zero) {
  extern __shared__ __align__(16) unsigned char smem[];
  FewShared<W>& sh = *reinterpret_cast<FewShared<W>*>(smem);
  const int tid = static_cast<int>(threadIdx.x), warp = tid / kWarp;
  const int lane = static_cast<int>(lane_id());
  grid_dependency_sync();
  // the list: words in ascending order, `size` of them, a power of two
  const int tokens = static_cast<int>(a.tokens);
  for (int i = tid; i < size; i += kFewThreads)
    sh.word[i] = i < tokens ? static_cast<W>(key_of(a, i)) << shift | static_cast<W>(i)
                            : ~static_cast<W>(0);
  __syncthreads();
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      for (int q = tid; q < size / 2; q += kFewThreads) {
        const int i = (q & ~(step - 1)) * 2 + (q & (step - 1)), j = i + step;
        const W x = sh.word[i], y = sh.word[j];
        if ((x > y) == ((i & run) == 0)) {
          sh.word[i] = y;
          sh.word[j] = x;
        }
      }
      // 64 neighbouring words are one warp's as long as steps stay inside
      if (step > kWarp || (step == 1 && run >= 2 * kWarp))
        __syncthreads();
      else
        __syncwarp();
    }
  __syncthreads();
  // its runs: the places where a live id differs from the one before
  constexpr int kEach = kFewTokens / kFewThreads;
  const int each = size > kFewThreads ? kEach : 1, base = tid * each;
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
  const uint32_t mine = static_cast<uint32_t>(__popc(heads)) << 16 | live;  // both at once
  uint32_t upto = mine;
#pragma unroll
  for (int o = 1; o < kWarp; o *= 2) {
    const uint32_t n = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += n;
  }
  if (lane == kWarp - 1) sh.part[warp] = upto;
  __syncthreads();
  uint32_t before = lane < kFewWarps ? sh.part[lane] : 0, all = before;
  before = __reduce_add_sync(kFull, lane < warp ? before : 0);
  all = __reduce_add_sync(kFull, all);
  const int runs = static_cast<int>(all >> 16);
  int run = static_cast<int>((before + upto - mine) >> 16);
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
  const int cta = static_cast<int>(blockIdx.x);
  if (cta >= sum_ctas) {
    const int64_t first = (cta - sum_ctas) * rows_per_zero;
    zero_rows<OUT>(a, sh.key, runs, first, min(first + rows_per_zero, a.vocab), 0.0f, sh.named);
    return;
  }
  const W places = (static_cast<W>(1) << shift) - 1;
  const int items = runs * blocks;
  auto row_of = [&](int r) { return a.mode == kEmbedRows ? static_cast<uint32_t>(r) : sh.key[r]; };
  for (int w = cta * kFewWarps + warp; w < items; w += sum_ctas * kFewWarps) {
    const int r = w / blocks, from = sh.start[r], to = sh.start[r + 1];
    const int64_t col = (static_cast<int64_t>(w - r * blocks) * kWarp + lane) * VEC;
    if (to - from > kLongRun || col >= a.width) continue;
    float sum[VEC];
    sum_rows<IN, VEC, W>(a, sh.word, places, from, to, col, sum);
    store_sum<IN, OUT, VEC>(a, row_of(r), col, sum);
  }
  // long runs, in as many parts as warps, joined in their order
  float* parts = reinterpret_cast<float*>(smem + sizeof(FewShared<W>));
  for (int w = cta; w < items; w += sum_ctas) {
    const int r = w / blocks, from = sh.start[r], to = sh.start[r + 1];
    if (to - from <= kLongRun) continue;
    const int64_t col = (static_cast<int64_t>(w - r * blocks) * kWarp + lane) * VEC;
    const int per = (to - from + kFewWarps - 1) / kFewWarps;
    float sum[VEC];
    if (col < a.width) {
      sum_rows<IN, VEC, W>(a, sh.word, places, min(from + warp * per, to),
                           min(from + (warp + 1) * per, to), col, sum);
#pragma unroll
      for (int i = 0; i < VEC; ++i) parts[(warp * VEC + i) * kWarp + lane] = sum[i];
    }
    __syncthreads();
    if (warp == 0 && col < a.width) {
      for (int n = 1; n < kFewWarps; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += parts[(n * VEC + i) * kWarp + lane];
      store_sum<IN, OUT, VEC>(a, row_of(r), col, sum);
    }
    __syncthreads();
  }
}

}  // namespace lsdrs
