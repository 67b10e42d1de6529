// sort_experts.cu — sort_by_expert: pairs of token and choice in the order of
// their experts.
//
// A counting sort in one launch. A warp takes neighbouring pairs, 32 at a time:
// lanes with the same expert find each other, their lowest counts them in the
// warp's own row of counters, so that ranks keep the pairs' order and nothing
// depends on the order of atomics. Counters become starts by sums over warps,
// over the blocks of a cluster (in shared memory), and over experts; the second
// pass hands out places.
//
// Few pairs take one block, many a cluster of eight.
#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_experts.h"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kThreads = 1024, kSortWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct SortParams {
  const int64_t* experts;
  int64_t* offsets;
  int64_t* rows;
  int64_t* places;
  int pairs, top_k, num_experts, blocks;
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t a, int rank) {
  uint32_t d, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(d) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1) sort_by_expert_kernel(const SortParams p) {
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t warp_sums[kSortWarps];
  uint32_t* const totals = sm;                     // of this block
  uint32_t* const counts = sm + p.num_experts;     // [warp][expert]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x;
  uint32_t* const mine = counts + warp * p.num_experts;
  for (int i = tid; i < kSortWarps * p.num_experts; i += kThreads) counts[i] = 0;
  __syncthreads();
  // this warp's pairs, a multiple of 32 but at the end
  const int warps = kSortWarps * p.blocks;
  const int per = (int)((((int64_t)p.pairs + warps - 1) / warps + 31) / 32 * 32);
  const int64_t first = (int64_t)(rank * kSortWarps + warp) * per;
  const int64_t last = first + per < p.pairs ? first + per : p.pairs;
  const auto expert = [&](int64_t i) -> uint32_t {
    if (i >= last) return kAll;
    const int64_t e = p.experts[i];
    return e >= 0 && e < p.num_experts ? (uint32_t)e : kAll;
  };
  for (int64_t i = first; i < last; i += 32) {
    const uint32_t e = expert(i + lane);
    const uint32_t same = __match_any_sync(kAll, e);
    if (e != kAll && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  uint32_t total = 0;
  if (tid < p.num_experts) {
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = counts[w * p.num_experts + tid];
      counts[w * p.num_experts + tid] = total;
      total += c;
    }
    totals[tid] = total;
  }
  uint32_t before = 0, of_all = total;
  if (p.blocks > 1) {
    cluster_sync();
    if (tid < p.num_experts) {
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(totals + tid);
      of_all = 0;
      for (int q = 0; q < p.blocks; ++q) {
        const uint32_t c = ld_cluster(at, q);
        before += q < rank ? c : 0;
        of_all += c;
      }
    }
  }
  // sum over the experts before
  uint32_t upto = of_all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  uint32_t start = upto - of_all;
  for (int w = 0; w < warp; ++w) start += warp_sums[w];
  if (tid < p.num_experts) {
    for (int w = 0; w < kSortWarps; ++w) counts[w * p.num_experts + tid] += start + before;
    if (rank == 0) p.offsets[tid] = start;
  }
  uint32_t placed = 0;
  for (int w = 0; w < kSortWarps; ++w) placed += warp_sums[w];
  if (rank == 0 && tid == 0) p.offsets[p.num_experts] = placed;
  __syncthreads();
  for (int64_t i = first; i < last; i += 32) {
    const uint32_t e = expert(i + lane);
    const uint32_t same = __match_any_sync(kAll, e);
    const uint32_t ahead = __popc(same & ((1u << lane) - 1u));
    const uint32_t place = e != kAll ? mine[e] + ahead : 0;
    __syncwarp();
    if (e != kAll && ahead == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i + lane < last) {
      p.places[i + lane] = e != kAll ? (int64_t)place : -1;
      if (e != kAll) p.rows[place] = (i + lane) / p.top_k;
    }
  }
  for (int64_t i = (int64_t)placed + rank * kThreads + tid; i < p.pairs; i += kThreads * p.blocks)
    p.rows[i] = -1;
  if (p.blocks > 1) cluster_sync();  // (its counts may still be read)
}

}  // namespace
}  // namespace kvq

extern "C" int sort_by_expert(const int64_t* experts, int64_t num_tokens, int64_t top_k,
                              int64_t num_experts, int64_t* offsets, int64_t* rows, int64_t* places,
                              cudaStream_t stream) {
  using namespace kvq;
  constexpr int64_t kMost = (1ll << 31) - 1024;
  if (num_tokens < 0 || num_tokens >= kMost || top_k < 1 || top_k >= kMost) return KVQ_EINVAL;
  if (num_tokens * top_k >= kMost || num_experts < 1 || num_experts > 1024) return KVQ_EINVAL;
  if (!offsets || !aligned(offsets, 8)) return KVQ_EINVAL;
  const bool any = num_tokens > 0;
  if ((any && (!experts || !rows || !places)) || !aligned(experts, 8) || !aligned(rows, 8) ||
      !aligned(places, 8))
    return KVQ_EINVAL;
  SortParams p;
  p.experts = experts;
  p.offsets = offsets;
  p.rows = rows;
  p.places = places;
  p.pairs = (int)(num_tokens * top_k);
  p.top_k = (int)top_k;
  p.num_experts = (int)num_experts;
  p.blocks = p.pairs > 4096 ? kCluster : 1;
  const size_t smem = (size_t)(kSortWarps + 1) * num_experts * 4;
  static int ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(sort_by_expert_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kSortWarps + 1) * 1024 * 4) != cudaSuccess) {
      cudaGetLastError();
      return KVQ_ECUDA;
    }
    ready[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.blocks > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, sort_by_expert_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  return launch_status();
}
