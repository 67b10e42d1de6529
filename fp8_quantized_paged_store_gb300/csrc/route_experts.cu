// route_experts.cu — route_experts: scores of the experts, the choice of the
// best, their weights.
//
//   score = softmax(x) or 1 / (1 + exp(-x)),  key = score + bias (x without a bias)
//   groups by the sum of their two largest, top_k by key, weights renormalised
//
// One warp takes a token, a lane E / 32 neighbouring experts, all in registers;
// a maximum over the warp is one reduction of ordered 32-bit keys, a second
// finds the lowest index among equals, so a choice costs two of them and a look
// over a lane's own experts.
//
// The choice has to be that of keys in binary64, which this GPU computes slowly:
// keys are formed in binary32 with a bound on their error, one place more than
// asked for is chosen, and only where two neighbours in the order lie within
// the bound are the keys of the experts in question formed again in binary64
// (about 1 token in 500). Without a bias the logits themselves are the keys and
// nothing is in question.
//
// Bound: few tokens by one warp's chain, many by its issue slots.
#include <cuda_fp16.h>

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_experts.h"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kLargest = 3.402823466e38f;

struct RouteParams {
  const uint8_t* logits;
  const float* bias;
  int64_t* experts;
  float* weights;
  int64_t tokens, pitch;  // bytes
  int num_experts, per;   // per lane
  int top_k, groups, top_groups, per_group;
  int dtype, sigmoid, renormalize;
  float scale;
};

__device__ __forceinline__ float logit_at(const RouteParams& p, const uint8_t* row, int e) {
  float x;
  if (p.dtype == KVQ_FP32)
    x = ld_f32(reinterpret_cast<const float*>(row) + e);
  else {
    uint16_t w;
    asm("ld.global.nc.u16 %0, [%1];" : "=h"(w) : "l"(row + 2 * e));
    x = p.dtype == KVQ_BF16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
  }
  // NaN is the lowest, infinity a number; -0 as +0, so that equal keys have equal bits
  x = x == x ? x : -INFINITY;
  return fminf(x, kLargest) + 0.0f;
}

// Bits ordered as the values are; 0 lies below every value.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) != 0 ? kAll : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) != 0 ? 0x80000000u : kAll));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The two largest of a pair's union.
template <typename T>
__device__ __forceinline__ void merge2(T& a, T& b, T c, T d) {
  const T top = a > c ? a : c, low = a > c ? c : a;
  const T second = a > c ? b : d;
  a = top;
  b = low > second ? low : second;
}

// Lane g's: the sum of the two largest of group g's keys, whose experts are
// neighbours; -inf for g >= groups. `slots`: the warp's, one for each expert.
template <typename T, int kPer>
__device__ __forceinline__ T group_value(const RouteParams& p, const T (&key)[kPer], T* slots,
                                         T lowest) {
  const int lane = threadIdx.x & 31;
  T value = lowest;
  if (p.num_experts % 32 == 0 && 32 % p.groups == 0) {
    // a group is 32 / groups whole lanes
    T a = lowest, b = lowest;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j < p.per) merge2(a, b, key[j], lowest);
    for (int o = 1; o < 32 / p.groups; o <<= 1) {
      const T c = __shfl_xor_sync(kAll, a, o), d = __shfl_xor_sync(kAll, b, o);
      merge2(a, b, c, d);
    }
    value = __shfl_sync(kAll, a + b, (lane * (32 / p.groups)) & 31);
    if (lane >= p.groups) value = lowest;
    return value;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * p.per + j;
    if (j < p.per && e < p.num_experts) slots[e] = key[j];
  }
  __syncwarp();
  if (lane < p.groups) {
    T a = lowest, b = lowest;
    for (int i = 0; i < p.per_group; ++i) merge2(a, b, slots[lane * p.per_group + i], lowest);
    value = a + b;
  }
  __syncwarp();
  return value;
}

// Bits of the top_groups groups of the largest values, lower indices first among
// equals; `gap`: between the last of them and the next.
template <typename T>
__device__ __forceinline__ uint32_t best_groups(const RouteParams& p, T value, T& gap) {
  const int lane = threadIdx.x & 31;
  int ahead = 0;
  for (int g = 0; g < p.groups; ++g) {
    const T v = __shfl_sync(kAll, value, g);
    ahead += v > value || (v == value && g < lane);
  }
  const bool in = lane < p.groups && ahead < p.top_groups;
  const uint32_t taken = __ballot_sync(kAll, in);
  const uint32_t last = __ballot_sync(kAll, lane < p.groups && ahead == p.top_groups - 1);
  const uint32_t next = __ballot_sync(kAll, lane < p.groups && ahead == p.top_groups);
  const T low = __shfl_sync(kAll, value, __ffs(last) - 1);
  const T high = __shfl_sync(kAll, value, next ? __ffs(next) - 1 : 0);
  gap = next ? low - high : (T)1e30;
  return taken;
}

template <int kPer>
__global__ void __launch_bounds__(32 * kWarps)
    route_experts_kernel(const RouteParams p) {
  extern __shared__ double shared_keys[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t >= p.tokens) return;
  double* const slots = shared_keys + warp * p.num_experts;
  const uint8_t* row = p.logits + t * p.pitch;

  float x[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * p.per + j;
    x[j] = j < p.per && e < p.num_experts ? logit_at(p, row, e) : -INFINITY;
  }
  float most = x[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) most = fmaxf(most, x[j]);
  most = from_ordered(__reduce_max_sync(kAll, ordered(most)));
  const bool none = most == -INFINITY;
  float total = 1.0f;
  const bool scores = p.bias || p.groups > 1;
  if (!p.sigmoid && (scores || !p.renormalize)) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += none ? 0.0f : expf(x[j] - most);
    total = warp_sum(sum);
  }
  const auto score_of = [&](float v) {
    if (p.sigmoid) return 1.0f / (1.0f + expf(-v));
    return none ? 0.0f : expf(v - most) / total;
  };
  // keys, and their distance from those in binary64: at most error * (1 + |key|)
  float key[kPer];
  if (scores) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane * p.per + j;
      const bool have = j < p.per && e < p.num_experts;
      key[j] = have ? score_of(x[j]) + (p.bias ? ld_f32(p.bias + e) : 0.0f) : -INFINITY;
    }
  }
  // sigmoid: exp, 1 + exp and the quotient, 8 halves of a step in all; softmax:
  // exp of a rounded difference (0.4), the sum of up to 1024 in 37 steps, the
  // quotient; the largest score is 1 / total
  const float error = 0x1p-24f * (1.0f + (p.sigmoid ? 8.0f : 64.0f / total));
  uint32_t groups = kAll;
  bool all = false;  // binary64 for every expert
  if (p.groups > 1) {
    float gap;
    const float value = group_value<float, kPer>(p, key, reinterpret_cast<float*>(slots), -INFINITY);
    groups = best_groups(p, value, gap);
    const float size = from_ordered(__reduce_max_sync(
        kAll, ordered(lane < p.groups && fabsf(value) < kLargest ? fabsf(value) : 0.0f)));
    all = !(gap > 4.0f * (error + 0x1p-23f * size));
  }
  const auto allowed = [&](int e, uint32_t taken) {
    return p.groups == 1 || (taken >> (e / p.per_group) & 1) != 0;
  };
  uint32_t u[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * p.per + j;
    const bool have = j < p.per && e < p.num_experts && allowed(e, groups);
    u[j] = have ? ordered(p.bias ? key[j] : x[j]) : 0u;
  }
  // the top_k, and one more to tell how near it comes
  int chosen = 0;  // lane i's: the i-th
  bool near = false;
  float before = 0.0f, size = 0.0f, least = 0.0f;
  const int places = p.bias ? p.top_k + 1 : p.top_k;
  for (int i = 0; i < places; ++i) {
    uint32_t top = u[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < kPer; ++j)
      if (u[j] > top) {
        top = u[j];
        at = j;
      }
    const uint32_t best = __reduce_max_sync(kAll, top);
    if (best == 0) break;  // (no expert beyond the top_k)
    const uint32_t e = __reduce_min_sync(kAll, top == best ? (uint32_t)(lane * p.per + at) : kAll);
    if (lane == i) chosen = (int)e;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (lane * p.per + j == (int)e) u[j] = 0u;
    if (p.bias) {
      const float k = from_ordered(best);
      size = fmaxf(size, fabsf(k));
      near = near || (i > 0 && !(before - k > 2.0f * (error + 0x1p-24f * size)));
      before = least = k;
    }
  }
  if (all || near) {
    // in binary64: the experts that may stand among the chosen, or all
    const float floor_key = least - 2.0f * (error + 0x1p-24f * size);
    double sum = 1.0;
    if (!p.sigmoid) {
      sum = 0.0;
#pragma unroll 1
      for (int j = 0; j < p.per; ++j) {
        const int e = lane * p.per + j;
        if (e < p.num_experts && !none) sum += exp((double)logit_at(p, row, e) - (double)most);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    double exact[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane * p.per + j;
      exact[j] = -INFINITY;
      if (j < p.per && e < p.num_experts && (all || (allowed(e, groups) && key[j] >= floor_key))) {
        const double v = x[j];
        const double s = p.sigmoid ? 1.0 / (1.0 + exp(-v)) : none ? 0.0 : exp(v - (double)most) / sum;
        exact[j] = p.bias ? s + (double)ld_f32(p.bias + e) : s;
      }
    }
    if (all) {
      double gap;
      groups = best_groups(p, group_value<double, kPer>(p, exact, slots, -INFINITY), gap);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane * p.per + j;
      const bool in = j < p.per && e < p.num_experts && allowed(e, groups) &&
                      (all || key[j] >= floor_key);
      if (!p.bias) exact[j] = x[j];
      u[j] = in;
    }
    for (int i = 0; i < p.top_k; ++i) {
      double top = -INFINITY;
      uint32_t e = kAll;  // (none; -inf is a key too)
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (u[j] && (e == kAll || exact[j] > top)) {
          top = exact[j];
          e = lane * p.per + j;
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double v = __shfl_xor_sync(kAll, top, o);
        const uint32_t f = __shfl_xor_sync(kAll, e, o);
        if (f != kAll && (e == kAll || v > top || (v == top && f < e))) {
          top = v;
          e = f;
        }
      }
      if (lane == i) chosen = (int)e;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lane * p.per + j == (int)e) u[j] = 0u;
    }
  }
  const bool mine = lane < p.top_k;
  float w = mine ? score_of(logit_at(p, row, chosen)) : 0.0f;
  if (p.renormalize) {
    const float sum = warp_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (mine) {
    p.experts[t * p.top_k + lane] = chosen;
    p.weights[t * p.top_k + lane] = w * p.scale;
  }
}

}  // namespace
}  // namespace kvq

extern "C" int route_experts(const void* logits, int64_t logit_stride, int32_t dtype,
                             int64_t num_tokens, int64_t num_experts, int64_t top_k, int32_t score,
                             const float* bias, int64_t groups, int64_t top_groups,
                             int32_t renormalize, float scale, int64_t* experts, float* weights,
                             cudaStream_t stream) {
  using namespace kvq;
  if (num_tokens < 0 || num_tokens > 0x7FFFFFFF) return KVQ_EINVAL;
  if (dtype != KVQ_BF16 && dtype != KVQ_FP16 && dtype != KVQ_FP32) return KVQ_EINVAL;
  if (score != KVQ_SOFTMAX && score != KVQ_SIGMOID) return KVQ_EINVAL;
  if (num_experts < 1 || num_experts > 1024 || groups < 1 || groups > 32 ||
      num_experts % groups || (groups > 1 && num_experts / groups < 2))
    return KVQ_EINVAL;
  if (top_groups < 1 || top_groups > groups) return KVQ_EINVAL;
  if (top_k < 1 || top_k > 32 || top_k > num_experts / groups * top_groups) return KVQ_EINVAL;
  if ((renormalize != 0 && renormalize != 1) || !(scale >= -3.4e38f && scale <= 3.4e38f))
    return KVQ_EINVAL;
  if (logit_stride < 0 || logit_stride > (1ll << 30)) return KVQ_EINVAL;
  if (num_tokens == 0) return KVQ_OK;
  const int size = dtype == KVQ_FP32 ? 4 : 2;
  if (!logits || !experts || !weights || !aligned(logits, size) || !aligned(bias, 4) ||
      !aligned(experts, 8) || !aligned(weights, 4))
    return KVQ_EINVAL;
  RouteParams p;
  p.logits = static_cast<const uint8_t*>(logits);
  p.bias = bias;
  p.experts = experts;
  p.weights = weights;
  p.tokens = num_tokens;
  p.pitch = logit_stride * size;
  p.num_experts = (int)num_experts;
  p.per = (int)((num_experts + 31) / 32);
  p.top_k = (int)top_k;
  p.groups = (int)groups;
  p.top_groups = (int)top_groups;
  p.per_group = (int)(num_experts / groups);
  p.dtype = dtype;
  p.sigmoid = score == KVQ_SIGMOID;
  p.renormalize = renormalize;
  p.scale = scale;
  // the groups' slow way needs a place for each expert
  const bool whole_lanes = num_experts % 32 == 0 && 32 % groups == 0;
  const size_t smem = groups > 1 && !whole_lanes ? (size_t)kWarps * num_experts * 8 : 0;
  const unsigned grid = (unsigned)((num_tokens + kWarps - 1) / kWarps);
  const auto launch = [&](auto kernel, int* ready) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
    if (smem > 48 * 1024 && !ready[dev]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536) !=
          cudaSuccess) {
        cudaGetLastError();
        return KVQ_ECUDA;
      }
      ready[dev] = 1;
    }
    kernel<<<grid, 32 * kWarps, smem, stream>>>(p);
    return launch_status();
  };
  static int ready[6][64];
  return p.per <= 1   ? launch(route_experts_kernel<1>, ready[0])
         : p.per <= 2 ? launch(route_experts_kernel<2>, ready[1])
         : p.per <= 4 ? launch(route_experts_kernel<4>, ready[2])
         : p.per <= 8 ? launch(route_experts_kernel<8>, ready[3])
         : p.per <= 16 ? launch(route_experts_kernel<16>, ready[4])
                       : launch(route_experts_kernel<32>, ready[5]);
}
