// K-EMBED: the plan of a gradient (tokens by id, as runs), dispatch by type and
// alignment, and the launches.
#include "embed.cuh"

#include <algorithm>

#include "kernels.h"

namespace lsdrs {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 4;
constexpr int kPlanTile = kPlanThreads * kPlanItems;

// A token's sort key: its id, or the table's length for one without a row.
__device__ __forceinline__ uint32_t key_of(const EmbedGradArgs& a, int64_t i) {
  const int64_t id = load_index(a.ids, a.index_bytes, i);
  return static_cast<uint32_t>(id < 0 || id >= a.vocab || id == a.padding_id ? a.vocab : id);
}

__global__ void __launch_bounds__(kPlanThreads)
    embed_keys_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p) {
  grid_dependency_sync();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  for (int64_t i = first; i < a.tokens; i += step) {
    p.keys[i] = key_of(a, i);
    p.vals[i] = static_cast<uint32_t>(i);
  }
  const int64_t words = static_cast<int64_t>(p.chunks) * p.blocks;
  for (int64_t i = first; i < words; i += step) p.scratch.arrived[i] = 0;
}

// Whether a run of live tokens begins at sorted place i.
__device__ __forceinline__ bool begins(const EmbedGradArgs& a, const uint32_t* keys, int64_t i) {
  return i < a.tokens && keys[i] < a.vocab && (i == 0 || keys[i] != keys[i - 1]);
}

__global__ void __launch_bounds__(kPlanThreads)
    embed_heads_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p) {
  __shared__ uint32_t part[kPlanThreads / kWarp];
  grid_dependency_sync();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanTile + threadIdx.x * kPlanItems;
  uint32_t n = 0;
#pragma unroll
  for (int u = 0; u < kPlanItems; ++u) n += begins(a, p.sorted_keys, first + u);
  n = __reduce_add_sync(kFull, n);
  if (lane_id() == 0) part[threadIdx.x / kWarp] = n;
  __syncthreads();
  if (threadIdx.x < kWarp) {
    n = __reduce_add_sync(kFull, part[threadIdx.x]);
    if (threadIdx.x == 0) p.tile_heads[blockIdx.x] = n;
  }
}

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* part) {
  v = __reduce_add_sync(kFull, v);
  __syncthreads();
  if (lane_id() == 0) part[threadIdx.x / kWarp] = v;
  __syncthreads();
  return __reduce_add_sync(kFull, part[lane_id()]);
}

__global__ void __launch_bounds__(kPlanThreads)
    embed_runs_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p) {
  static_assert(kPlanThreads == kWarp * kWarp);
  __shared__ uint32_t part[kWarp];
  grid_dependency_sync();
  // tokens that are not sorted are not looked at
  const bool failed = p.sort_error != nullptr && *p.sort_error != kErrNone;
  const int64_t tokens = failed ? 0 : a.tokens;
  // runs that begin in earlier tiles, and in all of them
  uint32_t before = 0, all = 0;
  for (unsigned t = threadIdx.x; t < gridDim.x; t += kPlanThreads) {
    const uint32_t n = p.tile_heads[t];
    all += n;
    if (t < blockIdx.x) before += n;
  }
  before = block_sum(before, part);
  all = block_sum(all, part);
  // and in this one, before this thread's places
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanTile + threadIdx.x * kPlanItems;
  bool head[kPlanItems];
  uint32_t n = 0;
#pragma unroll
  for (int u = 0; u < kPlanItems; ++u) {
    head[u] = begins(a, p.sorted_keys, first + u);
    n += head[u];
  }
  uint32_t upto = n;
#pragma unroll
  for (int o = 1; o < kWarp; o *= 2) {
    const uint32_t v = __shfl_up_sync(kFull, upto, o);
    if (lane_id() >= static_cast<uint32_t>(o)) upto += v;
  }
  __syncthreads();
  if (lane_id() == kWarp - 1) part[threadIdx.x / kWarp] = upto;
  __syncthreads();
  uint32_t run = before + upto - n +
                 __reduce_add_sync(kFull, lane_id() < threadIdx.x / kWarp ? part[lane_id()] : 0);
#pragma unroll
  for (int u = 0; u < kPlanItems; ++u) {
    const int64_t i = first + u;
    if (i >= tokens) break;
    const uint32_t key = p.sorted_keys[i];
    if (head[u]) {
      p.start[run] = static_cast<uint32_t>(i);
      p.key[run] = key;
      if (a.mode == kEmbedRows) a.row_ids[run] = key;
      ++run;
    }
    if (key < a.vocab) p.slot[i] = run - 1;
    // the live tokens end here
    const bool last = key < a.vocab && (i + 1 == a.tokens || p.sorted_keys[i + 1] >= a.vocab);
    if (last) {
      p.start[run] = static_cast<uint32_t>(i + 1);
      p.header[kRunsLive] = static_cast<uint32_t>(i + 1);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.header[kRunsCount] = all;
    p.header[kRunsFailed] = failed;
    if (failed && a.status != nullptr) *a.status = kErrLookback;
    if (all == 0) p.header[kRunsLive] = 0;
    if (a.mode == kEmbedRows) *a.count = static_cast<int>(all);
  }
  if (a.mode == kEmbedRows) {
    const int64_t rows = a.tokens < a.vocab ? a.tokens : a.vocab;
    for (int64_t i = all + static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; i < rows;
         i += static_cast<int64_t>(gridDim.x) * kPlanThreads)
      a.row_ids[i] = -1;
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(const void* p, int64_t stride, int64_t bytes, int es) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * es % bytes == 0;
}

// The widest access, in elements, that every row of both sides allows: 16
// bytes of the input, else 4, else one element.
int vector_of(int64_t width, int in_es, const void* in, int64_t in_stride, int out_es,
              const void* out, int64_t out_stride) {
  for (int vec : {16 / in_es, 4 / in_es})
    if (width % vec == 0 && aligned(in, in_stride, vec * in_es, in_es) &&
        aligned(out, out_stride, std::min(16, vec * out_es), out_es))
      return vec;
  return 1;
}

template <int TYPE, int VEC>
cudaError_t embed_as(const EmbedArgs& a, cudaStream_t s) {
  const int64_t per_row = a.width / VEC;
  const int64_t ctas = cdiv(a.tokens * per_row, kEmbedThreads * kEmbedBatch);
  return launch_kernel(embed_kernel<TYPE, VEC>, dim3(static_cast<unsigned>(ctas)),
                       dim3(kEmbedThreads), 0, s, a, static_cast<uint32_t>(per_row));
}

template <int TYPE>
cudaError_t embed_of(const EmbedArgs& a, cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<TYPE>::Raw);
  const int vec = vector_of(a.width, kEs, a.table, a.table_stride, kEs, a.out, a.out_stride);
  if (vec == 16 / kEs) return embed_as<TYPE, 16 / kEs>(a, s);
  if constexpr (kEs == 2)
    if (vec == 2) return embed_as<TYPE, 2>(a, s);
  return embed_as<TYPE, 1>(a, s);
}

int score_bytes(int type) { return type == RS_SCORE_F32 ? 4 : 2; }

// Scratch, every part 256-byte aligned.
struct Parts {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t was = at;
    at += align_up(bytes, 256);
    return was;
  }
};

int key_bits(int64_t vocab) {
  int bits = 1;
  while (vocab >> bits) ++bits;
  return bits;
}

// Lays a call's scratch out from `temp`; returns its size.
size_t lay_out(int64_t tokens, int64_t width, void* temp, GradPlan* p, size_t* sort) {
  Parts parts;
  unsigned char* base = static_cast<unsigned char*>(temp);
  auto words = [&](int64_t n) { return reinterpret_cast<uint32_t*>(base + parts.take(n * 4)); };
  const int64_t chunks = cdiv(tokens, kChunk);
  p->header = words(64);
  p->scratch.arrived = words(chunks * cdiv(width, kWarp));
  p->scratch.partial = reinterpret_cast<float*>(
      words(2 * chunks * static_cast<int64_t>(align_up(static_cast<size_t>(width), 256))));
  p->keys = words(tokens);
  p->vals = words(tokens);
  p->sorted_keys = words(tokens);
  p->pos = words(tokens);
  p->slot = p->keys;  // the unsorted tokens are done with
  p->key = p->vals;
  p->start = words(tokens + 1);
  p->tile_heads = words(cdiv(tokens, kPlanTile) + 1);
  p->chunks = static_cast<int>(chunks);
  *sort = parts.at;
  p->sort_error = tokens > 0 ? reinterpret_cast<const uint32_t*>(base + parts.at) : nullptr;
  return parts.at;
}

template <int IN, int OUT, int VEC>
cudaError_t grad_as(const EmbedGradArgs& a, GradPlan& p, int64_t sum_ctas, int64_t ctas,
                    cudaStream_t s) {
  return launch_kernel(embed_grad_kernel<IN, OUT, VEC>, dim3(static_cast<unsigned>(ctas)),
                       dim3(kGradThreads), 0, s, a, p, sum_ctas);
}

template <int IN, int OUT>
cudaError_t grad_of(const EmbedGradArgs& a, GradPlan& p, int vec, int64_t sum_ctas, int64_t ctas,
                    cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<IN>::Raw);
  if (vec == 16 / kEs) return grad_as<IN, OUT, 16 / kEs>(a, p, sum_ctas, ctas, s);
  if constexpr (kEs == 2)
    if (vec == 2) return grad_as<IN, OUT, 2>(a, p, sum_ctas, ctas, s);
  return grad_as<IN, OUT, 1>(a, p, sum_ctas, ctas, s);
}

}  // namespace

cudaError_t launch_embed(int type, const EmbedArgs& a, cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return embed_of<RS_SCORE_F16>(a, s);
    case RS_SCORE_BF16: return embed_of<RS_SCORE_BF16>(a, s);
    case RS_SCORE_F32: return embed_of<RS_SCORE_F32>(a, s);
  }
  return cudaErrorInvalidValue;
}

size_t embed_grad_temp(int64_t tokens, int64_t vocab, int64_t width) {
  GradPlan p{};
  size_t sort = 0;
  size_t total = lay_out(tokens, width, nullptr, &p, &sort);
  size_t sort_bytes = 0;
  if (tokens > 0 && radix_sort_keys_temp_bytes(static_cast<size_t>(tokens), 4, 4, 0,
                                               key_bits(vocab), 8, &sort_bytes) != RS_OK)
    return 0;
  return total + align_up(sort_bytes, 256);
}

cudaError_t launch_embed_keys(const EmbedGradArgs& a, cudaStream_t s) {
  GradPlan p{};
  size_t sort;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  p.blocks = static_cast<int>(cdiv(a.width, kWarp));  // any launch has no more
  const int64_t ctas = std::min<int64_t>(
      std::max<int64_t>(1, cdiv(a.tokens, kPlanThreads)), 4 * device_sm_count());
  return launch_kernel(embed_keys_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPlanThreads), 0,
                       s, a, p);
}

rs_status sort_embed_keys(const EmbedGradArgs& a, void* stream) {
  if (a.tokens == 0) return RS_OK;
  GradPlan p{};
  size_t sort, bytes = 0;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  const size_t n = static_cast<size_t>(a.tokens);
  const rs_status st = radix_sort_keys_temp_bytes(n, 4, 4, 0, key_bits(a.vocab), 8, &bytes);
  if (st != RS_OK) return st;
  return radix_sort_pairs_u32(p.keys, p.sorted_keys, p.vals, p.pos, n, 0, key_bits(a.vocab), 8,
                              static_cast<unsigned char*>(a.temp) + sort, bytes, stream);
}

cudaError_t launch_embed_runs(const EmbedGradArgs& a, int* launched, cudaStream_t s) {
  GradPlan p{};
  size_t sort;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  const dim3 tiles(static_cast<unsigned>(std::max<int64_t>(1, cdiv(a.tokens, kPlanTile))));
  const cudaError_t e = launch_kernel(embed_heads_kernel, tiles, dim3(kPlanThreads), 0, s, a, p);
  if (e != cudaSuccess) return e;
  *launched = 2;
  return launch_kernel(embed_runs_kernel, tiles, dim3(kPlanThreads), 0, s, a, p);
}

cudaError_t launch_embed_grad(int type, int out_type, const EmbedGradArgs& a, cudaStream_t s) {
  GradPlan p{};
  size_t sort;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  const int es = score_bytes(type), out_es = score_bytes(out_type);
  const int vec =
      vector_of(a.width, es, a.grad, a.grad_stride, out_es, a.out, a.out_stride);
  p.blocks = static_cast<int>(cdiv(a.width, static_cast<int64_t>(kWarp) * vec));
  p.piece = 128;
  static_assert(128 >= kChunk, "a chunk holds the beginnings of two pieces at most");
  const int64_t sum_ctas = cdiv(static_cast<int64_t>(p.chunks) * p.blocks, kGradWarps);
  p.rows_per_zero = std::min<int64_t>(kZeroMostRows, std::max<int64_t>(1, 131072 / (a.width * out_es)));
  const int64_t ctas = sum_ctas + (a.mode == kEmbedTable ? cdiv(a.vocab, p.rows_per_zero) : 0);
  if (ctas == 0) return cudaSuccess;
  if (type == RS_SCORE_F32) return grad_of<RS_SCORE_F32, RS_SCORE_F32>(a, p, vec, sum_ctas, ctas, s);
  if (type == RS_SCORE_F16)
    return out_type == RS_SCORE_F32
               ? grad_of<RS_SCORE_F16, RS_SCORE_F32>(a, p, vec, sum_ctas, ctas, s)
               : grad_of<RS_SCORE_F16, RS_SCORE_F16>(a, p, vec, sum_ctas, ctas, s);
  return out_type == RS_SCORE_F32
             ? grad_of<RS_SCORE_BF16, RS_SCORE_F32>(a, p, vec, sum_ctas, ctas, s)
             : grad_of<RS_SCORE_BF16, RS_SCORE_BF16>(a, p, vec, sum_ctas, ctas, s);
}

}  // namespace lsdrs
