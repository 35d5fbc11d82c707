// K-EMBED: the plan of a gradient (tokens by id, as runs), dispatch by type and
// alignment, and the launches.
#include "embed.cuh"

#include <algorithm>
#include <atomic>

#include "kernels.h"

namespace lsdrs {
namespace {

// ---- the list of up to kClusterTokens tokens, by one cluster
// 16 CTAs hold the tokens' (key, place) in shared memory and sort them there,
// digit by digit from the least: a warp ranks its 32 * ITEMS neighbouring words
// by ballots, the CTAs tell each other their digits' counts, and every word is
// written to its place in the CTA that this lies in: two passes of 9 bits for a
// vocabulary of 131,072, and 12 us for 8,191 tokens, 15 for 16,384, 19 for
// 32,768, bound by the latency of barriers and ranks.  The sort of whole keys
// takes 7 launches and 31 us for 16,384.  The gradient of 65,536 rows of 256
// takes 62 us this way, 72 that; of 100,000, with 8 words per thread, 82 and 78.
constexpr int kClusterCtas = 16;
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / kWarp;
constexpr int kClusterItems = 4;
constexpr int64_t kClusterTokens = int64_t(kClusterCtas) * kClusterThreads * kClusterItems;

struct ClusterShared {
  uint16_t warp_count[kClusterWarps][kMaxRadix];  // then: of the warps before
  uint32_t count[kClusterCtas][kMaxRadix];        // of each CTA
  uint32_t base[kMaxRadix];                       // where this CTA's words of a digit go
  uint32_t part[kWarp];
  // of each CTA: runs that begin there, its live tokens, and the list's place
  // of its first and last run (none: all ones, 0)
  uint4 ends[kClusterCtas];
};

__device__ __forceinline__ uint32_t cluster_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ uint32_t block_max_before(uint32_t v, uint32_t* part, uint32_t* all) {
  const uint32_t lane = lane_id(), warp = threadIdx.x / kWarp;
  uint32_t upto = v;
#pragma unroll
  for (int o = 1; o < kWarp; o *= 2) {
    const uint32_t n = __shfl_up_sync(kFull, upto, o);
    if (lane >= static_cast<uint32_t>(o)) upto = max(upto, n);
  }
  uint32_t before = __shfl_up_sync(kFull, upto, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  if (lane == kWarp - 1) part[warp] = upto;
  __syncthreads();
  const uint32_t n = part[lane];
  *all = __reduce_max_sync(kFull, n);
  return max(before, __reduce_max_sync(kFull, lane < warp ? n : 0));
}
__device__ __forceinline__ uint32_t block_min_after(uint32_t v, uint32_t* part, uint32_t* all) {
  const uint32_t lane = lane_id(), warp = threadIdx.x / kWarp;
  uint32_t from = v;
#pragma unroll
  for (int o = 1; o < kWarp; o *= 2) {
    const uint32_t n = __shfl_down_sync(kFull, from, o);
    if (lane + o < kWarp) from = min(from, n);
  }
  uint32_t after = __shfl_down_sync(kFull, from, 1);
  if (lane == kWarp - 1) after = 0xFFFFFFFFu;
  __syncthreads();
  if (lane == 0) part[warp] = from;
  __syncthreads();
  const uint32_t n = part[lane];
  *all = __reduce_min_sync(kFull, n);
  return min(after, __reduce_min_sync(kFull, lane > warp ? n : 0xFFFFFFFFu));
}

template <int ITEMS>
__global__ void __launch_bounds__(kClusterThreads, 1)
    embed_list_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p,
                      const int passes, const int bits) {
  constexpr uint32_t kSlice = kClusterThreads * ITEMS;  // words of a CTA
  extern __shared__ __align__(16) unsigned char smem[];
  uint64_t* word = reinterpret_cast<uint64_t*>(smem);
  ClusterShared& sh = *reinterpret_cast<ClusterShared*>(smem + kSlice * 8);
  const uint32_t tid = threadIdx.x, warp = tid / kWarp, lane = lane_id();
  const uint32_t rank = blockIdx.x;
  const uint32_t tokens = static_cast<uint32_t>(a.tokens), vocab = static_cast<uint32_t>(a.vocab);
  const uint32_t radix = 1u << bits;
  grid_dependency_sync();
  // (waited for before another CTA's memory is written to)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  uint64_t w[ITEMS];
  const uint32_t first = warp * kWarp * ITEMS + lane;  // this thread's words: every 32nd
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const uint32_t i = rank * kSlice + first + u * kWarp;
    // behind the last token: past every key
    w[u] = i < tokens ? static_cast<uint64_t>(key_of(a, i)) << 32 | i : ~uint64_t(0);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = 32 + pass * bits;
    uint32_t place[ITEMS];
    rank_words<ITEMS>(w, shift, bits, sh.warp_count[warp], place);
    __syncthreads();
    const uint32_t total = tid < radix ? sum_warps<kClusterWarps>(sh.warp_count, tid) : 0;
    if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid < radix)
#pragma unroll
      for (uint32_t r = 0; r < kClusterCtas; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                         cluster_peer(smem_addr(&sh.count[rank][tid]), r)),
                     "r"(total)
                     : "memory");
    cluster_barrier();
    uint32_t digit = 0, before = 0;
    if (tid < radix)
#pragma unroll
      for (uint32_t r = 0; r < kClusterCtas; ++r) {
        const uint32_t n = sh.count[r][tid];
        digit += n;
        if (r < rank) before += n;
      }
    uint32_t all;
    const uint32_t smaller = block_scan<kWarp>(digit, sh.part, &all);
    if (tid < radix) sh.base[tid] = smaller + before;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
      const uint32_t d = static_cast<uint32_t>(w[u] >> shift) & (radix - 1);
      const uint32_t to = sh.base[d] + sh.warp_count[warp][d] + place[u];
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                       cluster_peer(smem_addr(&word[to % kSlice]), to / kSlice)),
                   "l"(w[u])
                   : "memory");
    }
    cluster_barrier();
    if (pass + 1 < passes) {
#pragma unroll
      for (int u = 0; u < ITEMS; ++u) w[u] = word[first + u * kWarp];
    }
  }
  // the runs: ITEMS neighbouring words per thread
  const uint32_t base = tid * ITEMS, place0 = rank * kSlice + base;
  uint64_t last_word = 0;
  if (base > 0) {
    last_word = word[base - 1];
  } else if (rank > 0) {
    asm volatile("ld.shared::cluster.u64 %0, [%1];"
                 : "=l"(last_word)
                 : "r"(cluster_peer(smem_addr(&word[kSlice - 1]), rank - 1))
                 : "memory");
  }
  uint32_t heads = 0, live = 0, first_head = 0xFFFFFFFFu, last_head = 0;  // (places + 1)
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    w[u] = word[base + u];
    const uint32_t key = static_cast<uint32_t>(w[u] >> 32);
    const bool on = place0 + u < tokens && key < vocab;
    live += on;
    const uint64_t was = u == 0 ? last_word : w[u > 0 ? u - 1 : 0];
    if (on && (place0 + u == 0 || static_cast<uint32_t>(was >> 32) != key)) {
      heads |= 1u << u;
      first_head = min(first_head, place0 + u);
      last_head = place0 + u + 1;
    }
  }
  uint32_t all_heads, all_live, min_head, max_head;
  const uint32_t runs_before = block_scan<kWarp>(__popc(heads), sh.part, &all_heads);
  block_scan<kWarp>(live, sh.part, &all_live);
  uint32_t start = block_max_before(last_head, sh.part, &max_head);
  uint32_t end = block_min_after(first_head, sh.part, &min_head);
  if (tid < kClusterCtas) {
    const uint32_t to = cluster_peer(smem_addr(&sh.ends[rank]), tid);
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(all_heads),
                 "r"(all_live), "r"(min_head), "r"(max_head)
                 : "memory");
  }
  cluster_barrier();  // from here on no CTA reads another's memory
  // (written before, these words would be waited for at every barrier)
  const int64_t words = piece_places(a.tokens) * p.blocks;
  for (int64_t i = rank * kClusterThreads + tid; i < words; i += kClusterCtas * kClusterThreads)
    p.arrived[i] = 0;
  uint32_t run = runs_before, runs = 0, total_live = 0, next = 0xFFFFFFFFu;
  for (uint32_t r = 0; r < kClusterCtas; ++r) {
    const uint4 e = sh.ends[r];
    runs += e.x;
    total_live += e.y;
    if (r < rank) {
      run += e.x;
      start = max(start, e.w);  // (those of this CTA are larger, if any)
    }
    if (r > rank) next = min(next, e.z);
  }
  end = min(min(end, next), total_live);
  // ends from the right: of each word the next run's beginning
  uint32_t ends[ITEMS];
#pragma unroll
  for (int u = ITEMS - 1; u >= 0; --u) {
    ends[u] = end;
    if (heads >> u & 1) end = place0 + u;
  }
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const uint32_t i = place0 + u, key = static_cast<uint32_t>(w[u] >> 32);
    if (heads >> u & 1) {
      start = i + 1;
      p.key[run] = key;
      if (a.mode == kEmbedRows) a.row_ids[run] = key;
      ++run;
    }
    if (i < total_live)
      p.list[i] = Entry{static_cast<uint32_t>(w[u]), a.mode == kEmbedRows ? run - 1 : key,
                        start - 1, ends[u]};
  }
  if (rank == 0 && tid == 0) {
    p.header[kRunsCount] = runs;
    p.header[kRunsLive] = total_live;
    p.header[kRunsFailed] = 0;
    if (a.mode == kEmbedRows) *a.count = static_cast<int>(runs);
  }
  if (a.mode == kEmbedRows) {
    const int64_t rows = a.tokens < a.vocab ? a.tokens : a.vocab;
    for (int64_t i = runs + static_cast<int64_t>(rank * kClusterThreads + tid); i < rows;
         i += kClusterCtas * kClusterThreads)
      a.row_ids[i] = -1;
  }
}

// ---- the list of more tokens, by the sort of whole keys
constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 4;
constexpr int kPlanTile = kPlanThreads * kPlanItems;

__global__ void __launch_bounds__(kPlanThreads)
    embed_keys_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p) {
  grid_dependency_sync();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  for (int64_t i = first; i < a.tokens; i += step) {
    p.keys[i] = key_of(a, i);
    p.vals[i] = static_cast<uint32_t>(i);
  }
  const int64_t words = piece_places(a.tokens) * p.blocks;
  for (int64_t i = first; i < words; i += step) p.arrived[i] = 0;
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
  uint32_t n = 0, all;
#pragma unroll
  for (int u = 0; u < kPlanItems; ++u) n += begins(a, p.sorted_keys, first + u);
  block_scan<kWarp>(n, part, &all);
  if (threadIdx.x == 0) p.tile_heads[blockIdx.x] = all;
}

__global__ void __launch_bounds__(kPlanThreads)
    embed_runs_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ GradPlan p) {
  static_assert(kPlanThreads == kWarp * kWarp);
  __shared__ uint32_t part[kWarp];
  grid_dependency_sync();
  // tokens that are not sorted are not looked at
  const bool failed = *p.sort_error != kErrNone;
  const int64_t tokens = failed ? 0 : a.tokens;
  // runs that begin in earlier tiles, and in all of them
  uint32_t before = 0, all = 0;
  for (unsigned t = threadIdx.x; t < gridDim.x; t += kPlanThreads) {
    const uint32_t n = p.tile_heads[t];
    all += n;
    if (t < blockIdx.x) before += n;
  }
  block_scan<kWarp>(before, part, &before);
  block_scan<kWarp>(all, part, &all);
  if (failed) all = 0;
  // and in this one, before this thread's places
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanTile + threadIdx.x * kPlanItems;
  bool head[kPlanItems];
  uint32_t n = 0, tile;
#pragma unroll
  for (int u = 0; u < kPlanItems; ++u) {
    head[u] = begins(a, p.sorted_keys, first + u);
    n += head[u];
  }
  uint32_t run = before + block_scan<kWarp>(n, part, &tile);
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
    if (key < a.vocab && (i + 1 == a.tokens || p.sorted_keys[i + 1] >= a.vocab)) {
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

__global__ void __launch_bounds__(kPlanThreads)
    embed_entries_kernel(const __grid_constant__ EmbedGradArgs a,
                         const __grid_constant__ GradPlan p) {
  grid_dependency_sync();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  if (i >= p.header[kRunsLive]) return;
  const uint32_t slot = p.slot[i];
  p.list[i] = Entry{p.sorted_vals[i], a.mode == kEmbedRows ? slot : p.sorted_keys[i],
                    p.start[slot], p.start[slot + 1]};
}

constexpr int64_t kZeroFewBytes = 128 * 1024;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned(const void* p, int64_t stride, int64_t bytes, int es) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * es % bytes == 0;
}

// The widest access, in elements, that every row of both sides allows: `most`
// bytes of the input, 16, 4, or one element.
int vector_of(int most, int64_t width, int in_es, const void* in, int64_t in_stride, int out_es,
              const void* out, int64_t out_stride) {
  for (int vec : {most / in_es, 16 / in_es, 4 / in_es})
    if (width % vec == 0 && aligned(in, in_stride, vec * in_es, in_es) &&
        aligned(out, out_stride, std::min(32, vec * out_es), out_es))
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

template <int TYPE, int UNIT>
cudaError_t embed_narrow_as(const EmbedArgs& a, cudaStream_t s) {
  const int64_t blocks = cdiv(a.width, kWarp * kNarrow);
  const int64_t ctas = cdiv(a.tokens * blocks, kEmbedThreads / kWarp);
  return launch_kernel(embed_narrow_kernel<TYPE, UNIT>, dim3(static_cast<unsigned>(ctas)),
                       dim3(kEmbedThreads), 0, s, a, static_cast<uint32_t>(blocks));
}

template <int TYPE>
cudaError_t embed_of(const EmbedArgs& a, cudaStream_t s) {
  constexpr int kEs = sizeof(typename Score<TYPE>::Raw);
  const int vec = vector_of(32, a.width, kEs, a.table, a.table_stride, kEs, a.out, a.out_stride);
  if (vec == 32 / kEs) return embed_as<TYPE, 32 / kEs>(a, s);
  if (vec == 16 / kEs) return embed_as<TYPE, 16 / kEs>(a, s);
  if constexpr (kEs == 2)
    if (vec == 2) return embed_narrow_as<TYPE, 2>(a, s);
  return embed_narrow_as<TYPE, 1>(a, s);
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

// Lays a call's scratch out from `temp`; returns its size.  sort: where that of
// the sort of whole keys begins.
size_t lay_out(int64_t tokens, int64_t width, void* temp, GradPlan* p, size_t* sort) {
  Parts parts;
  unsigned char* base = static_cast<unsigned char*>(temp);
  auto words = [&](int64_t n) { return reinterpret_cast<uint32_t*>(base + parts.take(n * 4)); };
  p->header = words(64);
  *sort = parts.at;
  if (tokens <= kFewTokens) return parts.at;
  // Small ones, so that the last round of warps is short; of very many tokens
  // larger ones, which begin less often, if they make some rounds (bf16, chunks
  // of 8 and 32: 32,768 x 4,096 94 and 109 us, 65,536 x 2,048 103 and 115;
  // 200,000 x 1,024 155 and 148, 200,000 x 512 112 and 107).
  p->chunk = tokens <= kClusterTokens ? kLeastChunk : kMostChunk;
  while (p->chunk > kLeastChunk && tokens / p->chunk * cdiv(width, 512) < 5000) p->chunk /= 2;
  const int64_t chunks = cdiv(tokens, p->chunk);
  p->chunks = static_cast<int>(chunks);
  // an eighth of a 16-bit upstream gradient's size, and some
  const int64_t places = piece_places(tokens);
  p->arrived = words(places * cdiv(width, kLeastBlock));
  const size_t padded = align_up(static_cast<size_t>(width), width % 16 == 0 ? 512 : 256);
  p->partial = reinterpret_cast<float*>(words(places * static_cast<int64_t>(padded)));
  p->list = reinterpret_cast<Entry*>(words(tokens * 4));
  p->key = words(tokens);
  *sort = parts.at;
  if (tokens <= kClusterTokens) return parts.at;
  p->keys = words(tokens);
  p->vals = words(tokens);
  p->sorted_keys = words(tokens);
  p->sorted_vals = words(tokens);
  p->slot = p->keys;  // the unsorted tokens are done with
  p->start = words(tokens + 1);
  p->tile_heads = words(cdiv(tokens, kPlanTile));
  *sort = parts.at;
  p->sort_error = reinterpret_cast<const uint32_t*>(base + parts.at);
  return parts.at;
}

// One of the gradient's last kernels; f(types, elements of a lane, of an access).
template <int IN, int OUT, class F>
cudaError_t by_vector(int vec, const F& f) {
  constexpr int kEs = sizeof(typename Score<IN>::Raw);
  constexpr ScoreTag<IN> in{};
  constexpr ScoreTag<OUT> out{};
  if constexpr (F::kMost == 32)
    if (vec == 32 / kEs) return f(in, out, ScoreTag<32 / kEs>{}, ScoreTag<32 / kEs>{});
  if (vec == 16 / kEs) return f(in, out, ScoreTag<16 / kEs>{}, ScoreTag<16 / kEs>{});
  if constexpr (kEs == 2)
    if (vec == 2) return f(in, out, ScoreTag<kNarrow>{}, ScoreTag<2>{});
  return f(in, out, ScoreTag<kNarrow>{}, ScoreTag<1>{});
}
template <int MOST, class F>
struct UpTo : F {
  static constexpr int kMost = MOST;
};
template <int MOST, class F>
cudaError_t by_types(int type, int out_type, int vec, F&& launch) {
  const UpTo<MOST, F> f{launch};
  if (type == RS_SCORE_F32) return by_vector<RS_SCORE_F32, RS_SCORE_F32>(vec, f);
  if (type == RS_SCORE_F16)
    return out_type == RS_SCORE_F32 ? by_vector<RS_SCORE_F16, RS_SCORE_F32>(vec, f)
                                    : by_vector<RS_SCORE_F16, RS_SCORE_F16>(vec, f);
  return out_type == RS_SCORE_F32 ? by_vector<RS_SCORE_BF16, RS_SCORE_F32>(vec, f)
                                  : by_vector<RS_SCORE_BF16, RS_SCORE_BF16>(vec, f);
}

// Opts a kernel into its shared memory and clusters of 16, once per device.
template <class K>
cudaError_t allow(K kern, int bytes, std::atomic<uint64_t>* done) {
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

template <int ITEMS>
cudaError_t list_as(const EmbedGradArgs& a, const GradPlan& p, cudaStream_t s) {
  constexpr int kSmem = kClusterThreads * ITEMS * 8 + static_cast<int>(sizeof(ClusterShared));
  static_assert(kSmem <= 232448);
  static std::atomic<uint64_t> done{0};
  auto kern = embed_list_kernel<ITEMS>;
  const cudaError_t e = allow(kern, kSmem, &done);
  if (e != cudaSuccess) return e;
  const int bits = key_bits(a.vocab), passes = (bits + 8) / 9;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kClusterCtas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
#if LSDRS_PDL
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
#endif
  attr[n].id = cudaLaunchAttributeClusterDimension;
  attr[n].val.clusterDim.x = kClusterCtas;
  attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n + 1;
  return cudaLaunchKernelEx(&cfg, kern, a, p, passes, (bits + passes - 1) / passes);
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
  size_t sort = 0, sort_bytes = 0;
  const size_t total = lay_out(tokens, width, nullptr, &p, &sort);
  if (tokens > kClusterTokens &&
      radix_sort_keys_temp_bytes(static_cast<size_t>(tokens), 4, 4, 0, key_bits(vocab), 8,
                                 &sort_bytes) != RS_OK)
    return 0;
  return total + align_up(sort_bytes, 256);
}

bool embed_grad_sorts(int64_t tokens) { return tokens > kClusterTokens; }

cudaError_t launch_embed_keys(const EmbedGradArgs& a, cudaStream_t s) {
  GradPlan p{};
  size_t sort;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  p.blocks = static_cast<int>(cdiv(a.width, kLeastBlock));  // any launch has no more
  const int64_t ctas = std::min<int64_t>(cdiv(a.tokens, kPlanThreads), 4 * device_sm_count());
  return launch_kernel(embed_keys_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPlanThreads), 0,
                       s, a, p);
}

rs_status sort_embed_keys(const EmbedGradArgs& a, void* stream) {
  GradPlan p{};
  size_t sort, bytes = 0;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  const size_t n = static_cast<size_t>(a.tokens);
  const rs_status st = radix_sort_keys_temp_bytes(n, 4, 4, 0, key_bits(a.vocab), 8, &bytes);
  if (st != RS_OK) return st;
  return radix_sort_pairs_u32(p.keys, p.sorted_keys, p.vals, p.sorted_vals, n, 0,
                              key_bits(a.vocab), 8, static_cast<unsigned char*>(a.temp) + sort,
                              bytes, stream);
}

cudaError_t launch_embed_grad(int type, int out_type, const EmbedGradArgs& a, int* launched,
                              cudaStream_t s) {
  GradPlan p{};
  size_t sort;
  lay_out(a.tokens, a.width, a.temp, &p, &sort);
  const int es = score_bytes(type), out_es = score_bytes(out_type);
  const bool few = a.tokens <= kFewTokens;
  const int vec = vector_of(few ? 16 : 32, a.width, es, a.grad, a.grad_stride, out_es, a.out,
                            a.out_stride);
  const int64_t blocks = cdiv(a.width, kWarp * (vec * es >= 16 ? vec : kNarrow));
  const int sms = device_sm_count();
  if (few) {
    // every CTA sorts, so that there is one per SM for the sums; those of the zeros
    // only look which tokens are in their rows: four per SM, or 128 KB each (64
    // tokens into 131,072 x 1,024 f32 76 us, 80 with 512 KB; 1,500 into 32,000 x
    // 1,000 f16 21, 31 where they sorted too)
    const int64_t rows =
        std::min({static_cast<int64_t>(kZeroMostRows), cdiv(a.vocab, 4 * sms),
                  std::max<int64_t>(1, kZeroFewBytes / (a.width * out_es))});
    const int64_t sums =
        std::max<int64_t>(1, std::min<int64_t>(cdiv(a.tokens * blocks, kFewWarps), sms));
    int shift = 1;
    while (int64_t(1) << shift < a.tokens) ++shift;
    const int bits = key_bits(a.vocab), passes = (bits + 8) / 9;
    const dim3 ctas(
        static_cast<unsigned>(sums + (a.mode == kEmbedTable ? cdiv(a.vocab, rows) : 0)));
    return by_types<16>(type, out_type, vec, [&](auto in, auto out, auto v, auto unit) {
      auto go = [&](auto word) {
        using W = decltype(word);
        constexpr int kSmem = static_cast<int>(
            sizeof(FewShared<W>) + sizeof(Sum<decltype(v)::value>) * kFewThreads);
        static_assert(sizeof(FewShared<W>) % 8 == 0);
        static std::atomic<uint64_t> done{0};
        auto kern = embed_grad_few_kernel<decltype(in)::value, decltype(out)::value,
                                          decltype(v)::value, decltype(unit)::value, W>;
        if (kSmem > 48 * 1024) {
          const cudaError_t e = allow(kern, kSmem, &done);
          if (e != cudaSuccess) return e;
        }
        return launch_kernel(kern, ctas, dim3(kFewThreads), kSmem, s, a, shift, passes,
                             (bits + passes - 1) / passes, static_cast<int>(blocks),
                             static_cast<int>(sums), rows);
      };
      return key_bits(a.vocab) + shift <= 32 ? go(uint32_t{}) : go(uint64_t{});
    });
  }
  p.blocks = static_cast<int>(blocks);
  cudaError_t e = cudaSuccess;
  if (!embed_grad_sorts(a.tokens)) {
    const int64_t each = cdiv(a.tokens, kClusterCtas * kClusterThreads);
    static_assert(kClusterItems == 4);
    e = each <= 1   ? list_as<1>(a, p, s)
        : each <= 2 ? list_as<2>(a, p, s)
                    : list_as<4>(a, p, s);
    *launched = 2;
  } else {
    const dim3 tiles(static_cast<unsigned>(cdiv(a.tokens, kPlanTile)));
    e = launch_kernel(embed_heads_kernel, tiles, dim3(kPlanThreads), 0, s, a, p);
    if (e == cudaSuccess) e = launch_kernel(embed_runs_kernel, tiles, dim3(kPlanThreads), 0, s, a, p);
    if (e == cudaSuccess)
      e = launch_kernel(embed_entries_kernel,
                        dim3(static_cast<unsigned>(cdiv(a.tokens, kPlanThreads))),
                        dim3(kPlanThreads), 0, s, a, p);
    *launched = 4;
  }
  if (e != cudaSuccess) return e;
  const int64_t sum_ctas = cdiv(static_cast<int64_t>(p.chunks) * p.blocks, kGradWarps);
  p.rows_per_zero =
      std::min<int64_t>(kZeroMostRows, std::max<int64_t>(1, 131072 / (a.width * out_es)));
  const dim3 ctas(static_cast<unsigned>(
      sum_ctas +
      (a.mode == kEmbedTable ? cdiv(a.vocab, p.rows_per_zero) : 0)));
  return by_types<32>(type, out_type, vec, [&](auto in, auto out, auto v, auto unit) {
    return launch_kernel(
        embed_grad_kernel<decltype(in)::value, decltype(out)::value, decltype(v)::value,
                          decltype(unit)::value>,
        ctas, dim3(kGradThreads), 0, s, a, p, sum_ctas);
  });
}

}  // namespace lsdrs
