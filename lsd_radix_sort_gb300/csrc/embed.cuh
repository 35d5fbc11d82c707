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
// What the sort leaves: the live tokens' positions by id, as runs of equal ids.
struct Runs {
  const uint32_t* pos;     // positions, by run
  const uint32_t* slot;    // the run of each
  const uint32_t* start;   // of each run; one more: the number of live tokens
  const uint32_t* key;     // each run's id
  int runs, live;
};

// Work is dealt out in chunks of kChunk sorted tokens, a warp for each 32
// vectors of columns.  A warp adds up the runs that begin in its chunk, to
// their ends.  Runs of more than `piece` tokens are divided into such pieces,
// whose sums, in 32 bits, meet in scratch: whoever finishes a run's last
// piece adds them up, in their order.
constexpr int kChunk = 32;
constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / kWarp;
constexpr int kGradBatch = 8;

struct GradScratch {
  float* partial;       // [2 * chunks][padded width]: later pieces, first pieces
  uint32_t* arrived;    // [chunks][blocks]: pieces of the run that begins there
};

template <int IN, int OUT, int VEC>
__device__ __forceinline__ void store_sum(const EmbedGradArgs& a, int64_t row, int64_t col,
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

template <int IN, int OUT, int VEC>
__device__ __forceinline__ void sum_runs(const EmbedGradArgs& a, const Runs& r,
                                         const GradScratch& g, int chunk, int block, int blocks,
                                         int piece) {
  using P = Pack<IN, VEC>;
  using Raw = typename P::Raw;
  const int lane = static_cast<int>(lane_id());
  const int64_t col = (static_cast<int64_t>(block) * kWarp + lane) * VEC;
  const bool mine = col < a.width;
  const Raw* from = static_cast<const Raw*>(a.grad) + (mine ? col : 0);
  const int64_t padded = static_cast<int64_t>(blocks) * kWarp * VEC;
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  bool open = false;  // a piece is under way
  for (int window = chunk * kChunk; window < r.live; window += kChunk) {
    const int at = window + lane;
    const bool valid = at < r.live;
    const uint32_t slot = valid ? r.slot[at] : 0;
    const uint32_t pos = valid ? r.pos[at] : 0;
    const int start = valid ? static_cast<int>(r.start[slot]) : 0;
    const int end = valid ? static_cast<int>(r.start[slot + 1]) : 0;
    const uint32_t key = valid ? r.key[slot] : 0;
    const int off = at - start;
    const unsigned begins = __ballot_sync(kFull, valid && off % piece == 0);
    const unsigned ends = __ballot_sync(kFull, valid && (at + 1 == end || (off + 1) % piece == 0));
    int t, last;  // tokens [t, last) of the window are this warp's
    if (open) {   // what began before, to its end
      t = 0;
      last = ends != 0 ? __ffs(static_cast<int>(ends)) : kWarp;
    } else {
      if (begins == 0) return;
      t = __ffs(static_cast<int>(begins)) - 1;
      last = min(kWarp, r.live - window);
    }
    for (; t < last; t += kGradBatch) {
      P p[kGradBatch];
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        const uint32_t i = __shfl_sync(kFull, pos, min(t + u, kWarp - 1));
        p[u] = mine && t + u < last ? P::load(from + static_cast<int64_t>(i) * a.grad_stride)
                                    : P::zero();
      }
#pragma unroll
      for (int u = 0; u < kGradBatch; ++u) {
        if (t + u >= last) break;
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += p[u].get(i);
        if ((ends >> (t + u) & 1) == 0) continue;
        // the end of a run, or of a piece of one
        const int b = __shfl_sync(kFull, start, t + u), e = __shfl_sync(kFull, end, t + u);
        const uint32_t s = __shfl_sync(kFull, slot, t + u), k = __shfl_sync(kFull, key, t + u);
        const int64_t row = a.mode == kEmbedRows ? static_cast<int64_t>(s) : static_cast<int64_t>(k);
        bool whole = e - b <= piece;
        if (!whole) {
          const int pieces = (e - b + piece - 1) / piece;
          const int number = (window + t + u - b) / piece, first = b + number * piece;
          float* to = g.partial + (2 * (first / kChunk) + (number == 0)) * padded +
                      (static_cast<int64_t>(block) * kWarp + lane) * VEC;
          if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4)
              __stcg(reinterpret_cast<float4*>(to + i),
                     make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]));
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) __stcg(to + i, sum[i]);
          }
          __threadfence();
          __syncwarp();
          uint32_t before = 0;
          if (lane == 0)
            before = atomicAdd(&g.arrived[static_cast<int64_t>(b / kChunk) * blocks + block], 1u);
          before = __shfl_sync(kFull, before, 0);
          whole = static_cast<int>(before) == pieces - 1;
          if (whole) {  // every piece is there
            __threadfence();
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
            for (int n0 = 0; n0 < pieces; n0 += 4) {
              float v[4][VEC];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const float* part =
                    g.partial +
                    (2 * ((b + min(n0 + n, pieces - 1) * piece) / kChunk) + (n0 + n == 0)) * padded +
                    (static_cast<int64_t>(block) * kWarp + lane) * VEC;
                if constexpr (VEC % 4 == 0) {
#pragma unroll
                  for (int i = 0; i < VEC; i += 4) {
                    const float4 f = __ldcg(reinterpret_cast<const float4*>(part + i));
                    v[n][i] = f.x;
                    v[n][i + 1] = f.y;
                    v[n][i + 2] = f.z;
                    v[n][i + 3] = f.w;
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < VEC; ++i) v[n][i] = __ldcg(part + i);
                }
              }
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (n0 + n < pieces)
#pragma unroll
                  for (int i = 0; i < VEC; ++i) sum[i] += v[n][i];
            }
          }
        }
        if (whole && mine) store_sum<IN, OUT, VEC>(a, row, col, sum);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
      }
    }
    open = last == kWarp && (ends >> (kWarp - 1) & 1) == 0;
    if (!open) return;
  }
}

// Zeros (or `fill`) for the rows of the table [first, last) that no run names.
template <int OUT>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, const Runs& r, int64_t first,
                                          int64_t last, float fill, uint32_t* named) {
  using Raw = typename Score<OUT>::Raw;
  const Raw raw = Score<OUT>::store(fill);
  const uint32_t word = sizeof(Raw) == 4 ? raw : raw | static_cast<uint32_t>(raw) << 16;
  const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
  const int words = static_cast<int>((last - first + 31) / 32);
  for (int i = tid; i < words; i += kGradThreads) named[i] = 0;
  __syncthreads();
  // the first run of an id >= first: 32 places are looked up at a time
  int lo = 0, hi = r.runs;  // it is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + kWarp - 1) / kWarp;
    const int at = lo + lane * step;
    const unsigned below =
        __ballot_sync(kFull, at < hi && static_cast<int64_t>(r.key[at]) < first);
    const int n = __popc(below);  // places below: a prefix of them
    if (n == 0) break;
    const int left = lo + (n - 1) * step;
    hi = min(hi, left + step);
    lo = left + 1;
  }
  for (int i = lo + tid; i < r.runs; i += kGradThreads) {
    const int64_t v = static_cast<int64_t>(r.key[i]) - first;
    if (v >= last - first) break;
    atomicOr(&named[v / 32], 1u << (v % 32));
  }
  __syncthreads();
  const int warp = tid / kWarp;
  for (int64_t v = first + warp; v < last; v += kGradWarps) {
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

// What a call has laid out in its scratch; the header's words.
constexpr int kRunsCount = 0, kRunsLive = 1, kRunsFailed = 2;
struct GradPlan {
  uint32_t* header;
  const uint32_t* sort_error;  // the sort's device error word (null: no tokens)
  uint32_t *keys, *vals, *sorted_keys, *pos, *slot, *start, *key, *tile_heads;
  GradScratch scratch;
  int chunks, blocks, piece;
  int zero_ctas;
  int64_t rows_per_zero;
};

constexpr int kZeroMostRows = 4096;  // of one CTA

template <int IN, int OUT, int VEC>
__global__ void __launch_bounds__(kGradThreads)
    embed_grad_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p,
                      const int64_t sum_ctas) {
  __shared__ uint32_t named[kZeroMostRows / 32];
  grid_dependency_sync();
  Runs r{p.pos, p.slot, p.start, p.key, static_cast<int>(p.header[kRunsCount]),
         static_cast<int>(p.header[kRunsLive])};
  const int64_t cta = blockIdx.x;
  if (cta >= sum_ctas) {
    const int64_t first = (cta - sum_ctas) * p.rows_per_zero;
    zero_rows<OUT>(a, r, first, min(first + p.rows_per_zero, a.vocab),
                   p.header[kRunsFailed] != 0 ? NAN : 0.0f, named);
    return;
  }
  const int64_t w = cta * kGradWarps + threadIdx.x / kWarp;
  const int64_t chunk = w / p.blocks;
  if (chunk >= p.chunks) return;
  sum_runs<IN, OUT, VEC>(a, r, p.scratch, static_cast<int>(chunk), static_cast<int>(w % p.blocks),
                         p.blocks, p.piece);
}

}  // namespace lsdrs
