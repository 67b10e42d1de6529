// sort_experts.cu — sort_by_expert: pairs of token and choice in the order of
// their experts.
//
// A counting sort. A block takes neighbouring pairs, a warp neighbouring ones of these,
// 32 at a time: lanes with the same expert find each other, and the lowest counts them
// in the warp's own row of counters, so that ranks keep the pairs' order and nothing
// depends on the order of atomics. Counters become starts by sums over warps, over the
// blocks before, and over experts; a second pass hands out places.
//
// Few pairs take one block and one launch. For many, a first kernel leaves every block's
// counts in the workspace, and the second one's blocks, which begin beside it, add up those
// before them: 131,072 pairs of 256 experts by 128 blocks in 11.7 us; in one cluster of
// eight, with its counts in shared memory, they took 38, most of it stores of eight bytes
// to 32 places at once. 144 pairs of 64 experts: 4.1 us.
#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_experts.h"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kThreads = 1024, kSortWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;
// Pairs of one launch (2048 of 64 experts: 7.6 us, by two launches 8; 4096: 11 and 8.6), and
// blocks where there are more. (A block reads the counts of all blocks: with more pairs
// each has more of them.)
constexpr int64_t kFewPairs = 2048, kMostBlocks = 256;

struct SortParams {
  const int64_t* experts;
  int64_t* offsets;
  int64_t* rows;
  int64_t* places;
  uint32_t* counts;  // [block][expert]
  int pairs, top_k, num_experts, per;  // per: pairs of a warp, a multiple of 32
};

// A warp's pairs [first, last) and the expert of one.
struct Pairs {
  int64_t first, last;
};
__device__ __forceinline__ Pairs warp_pairs(const SortParams& p) {
  const int64_t first = ((int64_t)blockIdx.x * kSortWarps + (threadIdx.x >> 5)) * p.per;
  return {first, first + p.per < p.pairs ? first + p.per : p.pairs};
}
__device__ __forceinline__ uint32_t expert_of(const SortParams& p, const Pairs& w, int64_t i) {
  if (i >= w.last) return kAll;
  const int64_t e = p.experts[i];
  return e >= 0 && e < p.num_experts ? (uint32_t)e : kAll;
}

// Lanes' experts, and the lanes with the same one.
struct Match {
  uint32_t expert, same;
};

// Every warp's counts of its pairs; returns its last 32, the only ones of most warps.
__device__ __forceinline__ Match count_pairs(const SortParams& p, uint32_t* counts) {
  const int lane = threadIdx.x & 31;
  uint32_t* const mine = counts + (threadIdx.x >> 5) * p.num_experts;
  for (int i = threadIdx.x; i < kSortWarps * p.num_experts; i += kThreads) counts[i] = 0;
  __syncthreads();
  const Pairs w = warp_pairs(p);
  Match m = {kAll, 0};
  for (int64_t i = w.first; i < w.last; i += 32) {
    m.expert = expert_of(p, w, i + lane);
    m.same = __match_any_sync(kAll, m.expert);
    if (m.expert != kAll && lane == __ffs(m.same) - 1) mine[m.expert] += __popc(m.same);
    __syncwarp();
  }
  __syncthreads();
  return m;
}

__global__ void __launch_bounds__(kThreads, 1) count_by_expert_kernel(const SortParams p) {
  extern __shared__ uint32_t counts[];
  count_pairs(p, counts);
  for (int e = threadIdx.x; e < p.num_experts; e += kThreads) {
    uint32_t total = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) total += counts[w * p.num_experts + e];
    p.counts[(int64_t)blockIdx.x * p.num_experts + e] = total;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1) sort_by_expert_kernel(const SortParams p) {
  extern __shared__ uint32_t counts[];
  __shared__ uint32_t warp_sums[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Match last = count_pairs(p, counts);
  uint32_t total = 0, before = 0;
  if (tid < p.num_experts) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = counts[w * p.num_experts + tid];
      counts[w * p.num_experts + tid] = total;
      total += c;
    }
  }
  if (p.counts) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < p.num_experts) {
      total = 0;
#pragma unroll 16
      for (int q = 0; q < (int)gridDim.x; ++q) {
        const uint32_t c = p.counts[(int64_t)q * p.num_experts + tid];
        before += q < (int)blockIdx.x ? c : 0;
        total += c;
      }
    }
  }
  // sum over the experts before
  uint32_t upto = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(kAll, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  uint32_t start = upto - total, placed = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    start += w < warp ? warp_sums[w] : 0;
    placed += warp_sums[w];
  }
  if (tid < p.num_experts) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) counts[w * p.num_experts + tid] += start + before;
    if (blockIdx.x == 0) p.offsets[tid] = start;
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.num_experts] = placed;
  __syncthreads();
  uint32_t* const mine = counts + warp * p.num_experts;
  const Pairs w = warp_pairs(p);
  for (int64_t i = w.first; i < w.last; i += 32) {
    Match m = last;
    if (i + 32 < w.last) {
      m.expert = expert_of(p, w, i + lane);
      m.same = __match_any_sync(kAll, m.expert);
    }
    const uint32_t e = m.expert, same = m.same;
    const uint32_t ahead = __popc(same & ((1u << lane) - 1u));
    const uint32_t place = e != kAll ? mine[e] + ahead : 0;
    __syncwarp();
    if (e != kAll && ahead == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i + lane < w.last) {
      p.places[i + lane] = e != kAll ? (int64_t)place : -1;
      if (e != kAll) p.rows[place] = (uint32_t)(i + lane) / (uint32_t)p.top_k;
    }
  }
  for (int64_t i = (int64_t)placed + blockIdx.x * kThreads + tid; i < p.pairs;
       i += (int64_t)kThreads * gridDim.x)
    p.rows[i] = -1;
}

// Blocks for so many pairs: 1, or enough for a warp to have 32 at least.
int64_t sort_blocks(int64_t pairs) {
  if (pairs <= kFewPairs) return 1;
  const int64_t blocks = (pairs + kThreads - 1) / kThreads;
  return blocks < kMostBlocks ? blocks : kMostBlocks;
}

}  // namespace
}  // namespace kvq

extern "C" int64_t sort_by_expert_workspace_size(int64_t num_tokens, int64_t top_k,
                                                 int64_t num_experts) {
  constexpr int64_t kMost = (1ll << 31) - 1024;
  if (num_tokens < 0 || num_tokens >= kMost || top_k < 1 || top_k >= kMost) return KVQ_EINVAL;
  if (num_tokens * top_k >= kMost || num_experts < 1 || num_experts > 1024) return KVQ_EINVAL;
  const int64_t blocks = kvq::sort_blocks(num_tokens * top_k);
  return blocks > 1 ? blocks * num_experts * 4 : 0;
}

extern "C" int sort_by_expert(const int64_t* experts, int64_t num_tokens, int64_t top_k,
                              int64_t num_experts, int64_t* offsets, int64_t* rows, int64_t* places,
                              void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  using namespace kvq;
  const int64_t need = sort_by_expert_workspace_size(num_tokens, top_k, num_experts);
  if (need < 0 || !offsets || !aligned(offsets, 8)) return KVQ_EINVAL;
  const bool any = num_tokens > 0;
  if ((any && (!experts || !rows || !places)) || !aligned(experts, 8) || !aligned(rows, 8) ||
      !aligned(places, 8))
    return KVQ_EINVAL;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 4))) return KVQ_EINVAL;
  SortParams p;
  p.experts = experts;
  p.offsets = offsets;
  p.rows = rows;
  p.places = places;
  p.counts = need > 0 ? static_cast<uint32_t*>(workspace) : nullptr;
  p.pairs = (int)(num_tokens * top_k);
  p.top_k = (int)top_k;
  p.num_experts = (int)num_experts;
  const int64_t blocks = sort_blocks(p.pairs), warps = kSortWarps * blocks;
  p.per = (int)((p.pairs + warps - 1) / warps + 31) / 32 * 32;
  const size_t smem = (size_t)kSortWarps * num_experts * 4;
  static int ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(sort_by_expert_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortWarps * 1024 * 4) != cudaSuccess ||
        cudaFuncSetAttribute(count_by_expert_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortWarps * 1024 * 4) != cudaSuccess) {
      cudaGetLastError();
      return KVQ_ECUDA;
    }
    ready[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  if (p.counts && cudaLaunchKernelEx(&cfg, count_by_expert_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  // (the second kernel counts its own pairs while the first one's last blocks run)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.counts ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, sort_by_expert_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  return launch_status();
}
