// K-BALANCE: the counting launch and the dispatch by score type (one
// translation unit per type, compiled in parallel).
#include "balance.cuh"

namespace lsdrs {

namespace {

// One histogram of the ids per cluster: per CTA in shared memory, added up
// over the cluster through distributed shared memory.  No global atomics, so
// nothing has to be cleared beforehand.
__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const BalanceArgs a) {
  __shared__ int hist[RS_MAX_EXPERTS + 1];
  const int tid = static_cast<int>(threadIdx.x);
  for (int e = tid; e <= a.experts; e += kCountThreads) hist[e] = 0;
  __syncthreads();
  grid_dependency_sync();
  count_ids(a, hist, blockIdx.x * int64_t(kCountThreads) + tid, gridDim.x * int64_t(kCountThreads));
  bal_cluster_sync();
  const int rank = static_cast<int>(bal_cluster_rank());
  int* to = reinterpret_cast<int*>(static_cast<unsigned char*>(a.temp) +
                                   bal_header_bytes(a.experts)) +
            (blockIdx.x / kBalCluster) * (a.experts + 1);
  for (int e = rank * kCountThreads + tid; e <= a.experts; e += kBalCluster * kCountThreads)
    to[e] = cluster_count(hist, e, kBalCluster);
  if (blockIdx.x == 0) {  // what the second launch adds to
    BalHeader* head = static_cast<BalHeader*>(a.temp);
    if (tid == 0) head->ticket = head->nan = 0;
    for (int e = tid; e < a.experts; e += kCountThreads) head->sums[e] = 0;
  }
  bal_cluster_sync();  // no CTA ends while its histogram is read
}

}  // namespace

cudaError_t launch_balance_counts(const BalanceArgs& a, int clusters, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kBalCluster));
  cfg.blockDim = dim3(kCountThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
#if LSDRS_PDL
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
#endif
  attr[n].id = cudaLaunchAttributeClusterDimension;
  attr[n].val.clusterDim.x = kBalCluster;
  attr[n].val.clusterDim.y = 1;
  attr[n++].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, balance_count_kernel, a);
}

size_t balance_temp(int64_t tokens, int experts) {
  if (tokens * experts <= kBalSingle) return 0;
  return bal_header_bytes(experts) +
         align_up(static_cast<size_t>(kBalMaxHists) * (experts + 1) * sizeof(int), 256);
}

cudaError_t launch_balance_f16(LossMode, const BalanceArgs&, int*, cudaStream_t);
cudaError_t launch_balance_bf16(LossMode, const BalanceArgs&, int*, cudaStream_t);
cudaError_t launch_balance_f32(LossMode, const BalanceArgs&, int*, cudaStream_t);

cudaError_t launch_balance(int type, LossMode mode, const BalanceArgs& a, int* launched,
                           cudaStream_t s) {
  switch (type) {
    case RS_SCORE_F16: return launch_balance_f16(mode, a, launched, s);
    case RS_SCORE_BF16: return launch_balance_bf16(mode, a, launched, s);
    case RS_SCORE_F32: return launch_balance_f32(mode, a, launched, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace lsdrs
