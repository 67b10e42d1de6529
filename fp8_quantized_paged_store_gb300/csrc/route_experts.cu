// route_experts.cu — route_experts: scores of the experts, the choice of the
// best, their weights.
//
//   score = softmax(x) or 1 / (1 + exp(-x)),  key = score + bias (x without a bias)
//   groups by the sum of their two largest, top_k by key, weights renormalised
//
// One warp takes a token, a lane E / 32 neighbouring experts, all in registers. A lane
// keeps its three best; a choice is a maximum over the warp of ordered 32-bit keys and a
// vote for the lowest lane that has it, and only a lane whose three are gone looks over its
// experts again.
//
// The choice has to be that of keys in binary64, of which this GPU computes one for a
// warp in 60 cycles an operation: keys are formed in binary32 with a bound on their
// error, one place more than asked for is chosen, and where two neighbours in the order,
// or two groups at the border, lie within the bound (about 1 token in 500) the token is
// chosen again by keys in binary64 of the experts in question, one to a lane. Without a
// bias the logits themselves are the keys and nothing is in question but the groups.
//
// Bound: few tokens by one warp's chain (24 x 64 experts 2.8 us), many by comparisons and
// selections, about 1030 instructions a token of 256 experts: 16384 x 256 in 8 groups,
// sigmoid and bias, 20 us; without groups 18, without a bias either 11. Kernels of their
// own for whole lanes (kEven) took 3 us off the first.
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

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
  int vector;         // a lane's logits are one aligned piece of memory
  int slots;          // a warp's places in shared memory
  int group_shift;    // 1 << group_shift lanes are a group, -1: groups do not end with lanes
  uint32_t to_group;  // e * to_group >> 20 is e's group
  float scale;
};

// NaN is the lowest, infinity a number; -0 as +0, so that equal keys have equal bits.
__device__ __forceinline__ float tamed(float x) {
  x = x == x ? x : -INFINITY;
  return fminf(x, kLargest) + 0.0f;
}

__device__ __forceinline__ float widened(const RouteParams& p, uint32_t w) {
  return p.dtype == KVQ_BF16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half((uint16_t)w));
}

__device__ __forceinline__ float logit_at(const RouteParams& p, const uint8_t* row, int e) {
  if (p.dtype == KVQ_FP32) return tamed(ld_f32(reinterpret_cast<const float*>(row) + e));
  uint16_t w;
  asm("ld.global.nc.u16 %0, [%1];" : "=h"(w) : "l"(row + 2 * e));
  return tamed(widened(p, w));
}

// kN neighbouring values.
template <int kN>
__device__ __forceinline__ void load_floats(const float* from, float (&x)[kN]) {
  if constexpr (kN >= 4) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 v = ld_f4(from + i);
      x[i] = v.x;
      x[i + 1] = v.y;
      x[i + 2] = v.z;
      x[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = ld_f32(from + i);
  }
}

// A lane's logits, -inf behind the last expert.
template <int kPer, bool kEven>
__device__ __forceinline__ void load_logits(const RouteParams& p, const uint8_t* row, int lane,
                                            float (&x)[kPer]) {
  if (!kEven && !p.vector) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane * p.per + j;
      x[j] = j < p.per && e < p.num_experts ? logit_at(p, row, e) : -INFINITY;
    }
    return;
  }
  if (p.dtype == KVQ_FP32) {
    load_floats<kPer>(reinterpret_cast<const float*>(row) + lane * kPer, x);
  } else if constexpr (kPer == 1) {
    x[0] = logit_at(p, row, lane);
  } else {
    const uint8_t* from = row + lane * kPer * 2;
    uint32_t w[kPer / 2];
    if constexpr (kPer >= 8) {
#pragma unroll
      for (int i = 0; i < kPer / 8; ++i) {
        const uint4 v = ld_nc_v4(from + 16 * i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) w[i] = ld_u32(from + 4 * i);
    }
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      x[2 * i] = widened(p, w[i] & 0xFFFFu);
      x[2 * i + 1] = widened(p, w[i] >> 16);
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) x[j] = tamed(x[j]);
}

// Bits ordered as the values are; 0 lies below every value.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) != 0 ? kAll : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) != 0 ? 0x80000000u : kAll));
}
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x == 0.0 ? 0.0 : x);
  return u ^ ((u >> 63) != 0 ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ double from_ordered64(uint64_t u) {
  return __longlong_as_double((long long)(u ^ ((u >> 63) != 0 ? 1ull << 63 : ~0ull)));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  return from_ordered(__reduce_max_sync(kAll, ordered(v)));
}

// ------------------------------------------------------------------- keys ---

// Whether element j of a lane is an expert. kEven: every lane has kPer of them, in
// aligned pieces, and groups (if any) end with lanes.
template <bool kEven>
__device__ __forceinline__ bool is_expert(const RouteParams& p, int lane, int j) {
  return kEven || p.vector || (j < p.per && lane * p.per + j < p.num_experts);
}
template <bool kEven>
__device__ __forceinline__ int group_of(const RouteParams& p, int lane, int e) {
  return kEven || p.group_shift >= 0 ? lane >> p.group_shift : (int)((uint32_t)e * p.to_group >> 20);
}

// score + bias, -inf where there is no expert. Returns softmax's sum (1 for a sigmoid).
//
// Fast exponential and reciprocal: with d = |x| (softmax: the difference to the largest) the
// exponential is documented within 2 + 1.173 d units in the last place, (4 + 2.35 d) 2^-24
// relative. Sigmoid: times s (1 - s) that is 1.3 2^-24 at most, and 1 + exp and the
// reciprocal add 3 2^-24: key_error's 8 2^-24 hold. Softmax, with the difference's
// rounding: (4 + 3.35 d) e^-d <= 4, in 2^-24 of the largest score; of the sum of up to 1024 of
// these 19 at most (most of them at d = 5.5), its 36 roundings, the quotient's two: 61 in all,
// and 64 2^-24 of the largest score hold. What is less than binary32 holds (2^-126) is covered by
// key_error's 2^-24. The sum with the bias rounds once more, by 2^-24 of itself.
template <int kPer, bool kEven>
__device__ __forceinline__ float form_keys(const RouteParams& p, int lane, float most, bool none,
                                           const float (&x)[kPer], float (&key)[kPer]) {
  float total = 1.0f;
  if (p.sigmoid) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(key[j]) : "f"(1.0f + __expf(-x[j])));
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      key[j] = none ? 0.0f : __expf(x[j] - most);
      sum += key[j];
    }
    total = warp_sum(sum);
    const float by = none ? 0.0f : 1.0f / total;
#pragma unroll
    for (int j = 0; j < kPer; ++j) key[j] *= by;
  }
  if (p.bias) {
    if (kEven || p.vector) {
      float bias[kPer];
      load_floats<kPer>(p.bias + lane * kPer, bias);
#pragma unroll
      for (int j = 0; j < kPer; ++j) key[j] += bias[j];
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (is_expert<kEven>(p, lane, j)) key[j] += ld_f32(p.bias + lane * p.per + j);
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (!is_expert<kEven>(p, lane, j)) key[j] = -INFINITY;
  return total;
}
__device__ __forceinline__ float key_error(const RouteParams& p, float total) {
  return 0x1p-24f * (1.0f + (p.sigmoid ? 8.0f : 64.0f / total));
}

// The two largest of a pair's union.
template <typename T>
__device__ __forceinline__ void merge2(T& a, T& b, T c, T d) {
  const T top = a > c ? a : c, low = a > c ? c : a;
  const T second = a > c ? b : d;
  a = top;
  b = low > second ? low : second;
}

// Lane g's: the two largest of group g's keys, whose experts are neighbours; -inf for g
// >= groups. `slots`: the warp's, one for each expert.
template <typename T>
struct Two {
  T x, y;
};
template <typename T, int kPer, bool kEven>
__device__ __forceinline__ Two<T> group_two(const RouteParams& p, const T (&key)[kPer], T* slots) {
  const int lane = threadIdx.x & 31;
  const T lowest = (T)-INFINITY;
  T a = lowest, b = lowest;
  if (kEven || p.group_shift >= 0) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (kEven || p.vector || j < p.per) merge2(a, b, key[j], lowest);
    for (int o = 1; o < 1 << p.group_shift; o <<= 1) {
      const T c = __shfl_xor_sync(kAll, a, o), d = __shfl_xor_sync(kAll, b, o);
      merge2(a, b, c, d);
    }
    a = __shfl_sync(kAll, a, (lane << p.group_shift) & 31);
    b = __shfl_sync(kAll, b, (lane << p.group_shift) & 31);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (is_expert<kEven>(p, lane, j)) slots[lane * p.per + j] = key[j];
    __syncwarp();
    if (lane < p.groups)
      for (int i = 0; i < p.per_group; ++i) merge2(a, b, slots[lane * p.per_group + i], lowest);
    __syncwarp();
  }
  return lane < p.groups ? Two<T>{a, b} : Two<T>{lowest, lowest};
}

// Bits of the top_groups groups of the largest values, lower indices first among
// equals; `last` and `next`: the value of the last of them and of the one behind it.
template <typename T>
__device__ __forceinline__ uint32_t best_groups(const RouteParams& p, T value, T& last, T& next) {
  const int lane = threadIdx.x & 31;
  int ahead = 0;
  for (int g = 0; g < p.groups; ++g) {
    const T v = __shfl_sync(kAll, value, g);
    ahead += v > value || (v == value && g < lane);
  }
  const bool in = lane < p.groups;
  const uint32_t taken = __ballot_sync(kAll, in && ahead < p.top_groups);
  const uint32_t low = __ballot_sync(kAll, in && ahead == p.top_groups - 1);
  const uint32_t high = __ballot_sync(kAll, in && ahead == p.top_groups);
  last = __shfl_sync(kAll, value, __ffs(low) - 1);
  next = high ? __shfl_sync(kAll, value, __ffs(high) - 1) : (T)-INFINITY;
  return taken;
}

// Half a group's value, which binary32 holds whatever the keys are, and how far two of these may
// stand the wrong way round: the value's error is that of its two keys, key_error's and 2^-24 of
// each, and the sum's, 2^-24 of itself. It goes by the keys, which may be far larger than a value
// in which they nearly cancel.
__device__ __forceinline__ float half_value(const Two<float>& two) { return 0.5f * two.x + 0.5f * two.y; }
__device__ __forceinline__ float group_error(const Two<float>& two, float error) {
  const float x = fabsf(two.x), y = fabsf(two.y);
  return 2.0f * error + warp_max((x <= kLargest ? 0x1p-22f * x : 0.0f) + (y <= kLargest ? 0x1p-22f * y : 0.0f));
}

// The first `places` of ordered keys (0: none) by the warp; lane i gets the i-th expert and
// its key. The lowest of the lanes with the largest key, whose experts are neighbours, has
// the lowest index.
struct Choice {
  int expert;
  uint32_t key, last;  // last: of the last place there is
  int found;           // places there are
};
template <int kPer>
__device__ __forceinline__ Choice choose(const RouteParams& p, const uint32_t (&u)[kPer], int places) {
  const int lane = threadIdx.x & 31;
  // a lane's three largest behind its last choice (key `past`, element `past_at`)
  uint32_t first = 0, second = 0, third = 0, past = kAll;
  int first_at = 0, second_at = 0, third_at = 0, past_at = -1;
  Choice c = {0, 0, 0, 0};
  const auto look = [&](auto again) {
    first = second = third = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t k = !decltype(again)::value || u[j] < past || (u[j] == past && j > past_at) ? u[j] : 0u;
      const bool best = k > first, good = k > second, fair = k > third;
      third = good ? second : fair ? k : third;
      third_at = good ? second_at : fair ? j : third_at;
      second = best ? first : good ? k : second;
      second_at = best ? first_at : good ? j : second_at;
      first = best ? k : first;
      first_at = best ? j : first_at;
    }
  };
  look(std::false_type{});
  for (; c.found < places; ++c.found) {
    const uint32_t best = __reduce_max_sync(kAll, first);
    if (best == 0) break;  // (no expert beyond the top_k)
    const int source = __ffs(__ballot_sync(kAll, first == best)) - 1;
    const int e = __shfl_sync(kAll, lane * p.per + first_at, source);
    if (lane == c.found) {
      c.expert = e;
      c.key = best;
    }
    c.last = best;
    if (lane == source) {
      past = first;
      past_at = first_at;
      first = second;
      first_at = second_at;
      second = third;
      second_at = third_at;
      third = 0;
      if (first == 0) look(std::true_type{});
    }
  }
  return c;
}

// ------------------------------------------------------ keys in binary64 ---

// The key of this lane's expert (-1: none) in binary64, as ordered bits; 0 without one.
// The whole warp. (Small functions apart: a token in 500 comes here, to instructions that
// no cache holds.)
__device__ __noinline__ uint64_t exact_key(const RouteParams& p, const uint8_t* row, int expert,
                                           float most, bool none) {
  double sum = 1.0;
  if (!p.sigmoid) {
    sum = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < p.num_experts; e += 32)
      if (!none) sum += exp((double)logit_at(p, row, e) - (double)most);
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  }
  if (expert < 0) return 0;
  const double v = logit_at(p, row, expert);
  const double t = exp(p.sigmoid ? -v : v - (double)most);
  const double s = !p.sigmoid && none ? 0.0 : (p.sigmoid ? 1.0 : t) / (p.sigmoid ? 1.0 + t : sum);
  return ordered64(p.bias ? s + (double)ld_f32(p.bias + expert) : s);
}

// Lane i's: the i-th of `count` experts, one to a lane, in the order of their keys.
__device__ __noinline__ int order_exactly(const RouteParams& p, const uint8_t* row, int* slots,
                                          int expert, int count, float most, bool none) {
  const int lane = threadIdx.x & 31;
  const uint64_t mine = exact_key(p, row, expert, most, none);
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const uint64_t k = __shfl_sync(kAll, mine, i);
    const int e = __shfl_sync(kAll, expert, i);
    rank += k > mine || (k == mine && e < expert);
  }
  if (expert >= 0) slots[rank] = expert;
  __syncwarp();
  const int ordered = slots[lane];
  __syncwarp();
  return ordered;
}

// Bits of the groups that stay. Lane g's `side`: 1 for a group above the border, -1 below
// it, 0 for one at it, whose value is formed of the two largest keys of its experts among
// `count` of them, one to a lane.
__device__ __noinline__ uint32_t groups_exactly(const RouteParams& p, const uint8_t* row, int expert,
                                                int count, int side, float most, bool none) {
  const int lane = threadIdx.x & 31;
  const uint64_t mine = exact_key(p, row, expert, most, none);
  uint64_t a = 0, b = 0;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const uint64_t k = __shfl_sync(kAll, mine, i);
    const int e = __shfl_sync(kAll, expert, i);
    if (e / p.per_group == lane) merge2<uint64_t>(a, b, k, 0);
  }
  const uint64_t value = side > 0 ? ~0ull : side < 0 ? 0 : ordered64(from_ordered64(a) + from_ordered64(b));
  int ahead = 0;
#pragma unroll 1
  for (int g = 0; g < p.groups; ++g) {
    const uint64_t v = __shfl_sync(kAll, value, g);
    ahead += v > value || (v == value && g < lane);
  }
  return __ballot_sync(kAll, lane < p.groups && ahead < p.top_groups);
}

// The choice by keys in binary64 of every expert, for a token with more than 32 of them
// in question (many equal keys).
template <int kPer>
__device__ __noinline__ int choose_exactly(const RouteParams& p, const uint8_t* row, double* slots,
                                           float most, bool none) {
  const int lane = threadIdx.x & 31;
  double sum = 1.0;
  if (!p.sigmoid) {
    sum = 0.0;
#pragma unroll 1
    for (int j = 0; j < p.per; ++j)
      if (is_expert<false>(p, lane, j) && !none)
        sum += exp((double)logit_at(p, row, lane * p.per + j) - (double)most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  }
  uint32_t groups = kAll;
  double exact[kPer];
#pragma unroll 1
  for (int j = 0; j < kPer; ++j) {
    exact[j] = -INFINITY;
    if (is_expert<false>(p, lane, j)) {
      const double v = logit_at(p, row, lane * p.per + j);
      const double s = p.sigmoid ? 1.0 / (1.0 + exp(-v)) : none ? 0.0 : exp(v - (double)most) / sum;
      exact[j] = p.bias ? s + (double)ld_f32(p.bias + lane * p.per + j) : s;
    }
  }
  if (p.groups > 1) {
    const Two<double> two = group_two<double, kPer, false>(p, exact, slots);
    double unused, too;
    groups = best_groups(p, lane < p.groups ? two.x + two.y : (double)-INFINITY, unused, too);
  }
  uint32_t left = 0;
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * p.per + j;
    if (is_expert<false>(p, lane, j) && (groups >> group_of<false>(p, lane, e) & 1) != 0) left |= 1u << j;
    if (!p.bias && is_expert<false>(p, lane, j)) exact[j] = logit_at(p, row, e);
  }
  int chosen = 0;
  for (int i = 0; i < p.top_k; ++i) {
    double top = -INFINITY;
    uint32_t e = kAll;  // (none; -inf is a key too)
    for (int j = 0; j < kPer; ++j)
      if ((left >> j & 1) != 0 && (e == kAll || exact[j] > top)) {
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
    if (e / p.per == lane) left &= ~(1u << (e - lane * p.per));
  }
  return chosen;
}

// ---------------------------------------------------------------- weights ---

// A chosen score below kSmall, of a logit that binary64 tells from nothing, and all weights of
// its token are formed in binary64: of what binary32 has left of such scores, a quotient or a
// large scale would make wrong weights. (Real routers' scores hardly come here.)
constexpr float kSmall = 0x1p-100f, kNothing = -746.0f;
__device__ __noinline__ float small_weight(const RouteParams& p, float v, float most, float total) {
  double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)most) / total;
  if (p.renormalize) {
    double sum = s;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  return (float)(s * p.scale);
}

// ----------------------------------------------------------------- kernel ---

// kPlain: neither bias nor groups, the logits are the keys.
template <int kPer, bool kPlain, bool kEven>
__global__ void __launch_bounds__(32 * kWarps, kPer <= 8 ? 4 : kPer <= 16 ? 3 : 2)
    route_experts_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ double shared_keys[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t >= p.tokens) return;
  const uint8_t* row = p.logits + t * p.pitch;

  float x[kPer];
  load_logits<kPer, kEven>(p, row, lane, x);
  float most = x[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) most = fmaxf(most, x[j]);
  most = warp_max(most);
  const bool none = most == -INFINITY;
  float total = 1.0f;
  int chosen;
  uint32_t u[kPer];
  if constexpr (kPlain) {
    if (!p.sigmoid && !p.renormalize) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum += none ? 0.0f : __expf(x[j] - most);
      total = warp_sum(sum);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) u[j] = is_expert<kEven>(p, lane, j) ? ordered(x[j]) : 0u;
    chosen = choose<kPer>(p, u, p.top_k).expert;
  } else {
    float key[kPer];
    total = form_keys<kPer, kEven>(p, lane, most, none, x, key);
    const float error = key_error(p, total);
    double* const slots = shared_keys + warp * p.slots;
    uint32_t groups = kAll;
    bool near = false, many = false;  // (many: more than 32 experts in question)
    // Experts of which `in` tells, one to a lane; -1: none.
    int* const list = reinterpret_cast<int*>(slots);
    int count = 0;
    const auto listed = [&](auto in) {
      count = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool take = in(j);
        const uint32_t m = __ballot_sync(kAll, take);
        const int at = count + __popc(m & ((1u << lane) - 1u));
        if (take && at < 32) list[at] = lane * p.per + j;
        count += __popc(m);
      }
      __syncwarp();
      const int expert = lane < count ? list[lane] : -1;
      __syncwarp();
      return expert;
    };
    if (p.groups > 1) {
      float last, next;
      const Two<float> two = group_two<float, kPer, kEven>(p, key, reinterpret_cast<float*>(slots));
      const float value = lane < p.groups ? half_value(two) : -INFINITY;
      groups = best_groups(p, value, last, next);
      const float off = group_error(two, error);
      if (!(last - next > off)) {
        // groups next to the border by their exact values: of each, what may be its two largest
        const int side = value > last + off ? 1 : lane < p.groups && value >= next - off ? 0 : -1;
        const uint32_t borders = __ballot_sync(kAll, side == 0);
        const float least = two.y - off;
        const int expert = listed([&](int j) {
          const bool have = is_expert<kEven>(p, lane, j);
          const int g = have ? group_of<kEven>(p, lane, lane * p.per + j) : 0;
          const float of_group = __shfl_sync(kAll, least, g);
          return have && (borders >> g & 1) != 0 && key[j] >= of_group;
        });
        if (count <= 32)
          groups = groups_exactly(p, row, expert, count, side, most, none);
        else
          many = true;
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool in = is_expert<kEven>(p, lane, j) && (groups >> group_of<kEven>(p, lane, lane * p.per + j) & 1) != 0;
      u[j] = in ? ordered(p.bias ? key[j] : x[j]) : 0u;
    }
    // one more than the top_k, to tell how near it comes
    const Choice c = choose<kPer>(p, u, p.bias ? p.top_k + 1 : p.top_k);
    chosen = c.expert;
    const float before = from_ordered(c.last);
    float size = 0.0f;
    if (p.bias) {
      const float k = from_ordered(c.key), below = __shfl_down_sync(kAll, k, 1);
      const float next = lane == 31 ? before : below;
      if (lane < c.found && fabsf(k) <= kLargest) size = fabsf(k);
      if (fabsf(before) <= kLargest) size = fmaxf(size, fabsf(before));
      size = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
      near = __any_sync(kAll, lane + 1 < c.found && !(k - next > 2.0f * (error + 0x1p-24f * size)));
    }
    if (near && !many) {
      // the experts that may stand among the chosen
      const uint32_t least = ordered(before - 2.0f * (error + 0x1p-24f * size));
      const int expert = listed([&](int j) { return u[j] != 0 && u[j] >= least; });
      if (count <= 32)
        chosen = order_exactly(p, row, list, expert, count, most, none);
      else
        many = true;
    }
    if (many) chosen = choose_exactly<kPer>(p, row, slots, most, none);
  }
  const bool mine = lane < p.top_k;
  float v = -INFINITY, w = 0.0f;
  if (mine) {
    chosen = min(max(chosen, 0), p.num_experts - 1);  // (a bias of NaN or infinity leaves any)
    v = logit_at(p, row, chosen);
    w = p.sigmoid ? 1.0f / (1.0f + expf(-v)) : none ? 0.0f : expf(v - most) / total;
  }
  if (__any_sync(kAll, w < kSmall && v - (p.sigmoid ? 0.0f : most) > kNothing)) {
    w = small_weight(p, v, most, total);
  } else {
    if (p.renormalize) {
      const float sum = warp_sum(w);
      w = sum > 0.0f ? w / sum : 0.0f;
    }
    w *= p.scale;
  }
  if (mine) {
    p.experts[t * p.top_k + lane] = chosen;
    p.weights[t * p.top_k + lane] = w;
  }
}

template <int kPer>
int launch(const RouteParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)kWarps * p.slots * 8;
  const bool plain = !p.bias && p.groups == 1;
  const bool even = p.vector && p.per == kPer && (p.groups == 1 || p.group_shift >= 0);
  const auto kernel = plain ? even ? route_experts_kernel<kPer, true, true>
                                   : route_experts_kernel<kPer, true, false>
                      : even ? route_experts_kernel<kPer, false, true>
                             : route_experts_kernel<kPer, false, false>;
  if (smem > 48 * 1024) {
    static int ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(route_experts_kernel<kPer, false, false>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, 65536) != cudaSuccess) {
        cudaGetLastError();
        return KVQ_ECUDA;
      }
      ready[dev] = 1;
    }
  }
  kernel<<<(unsigned)((p.tokens + kWarps - 1) / kWarps), 32 * kWarps, plain ? 0 : smem, stream>>>(p);
  return launch_status();
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
  p.group_shift = -1;
  if (num_experts % 32 == 0)
    for (int s = 0; s <= 5; ++s)
      if (groups << s == 32) p.group_shift = s;
  p.to_group = (uint32_t)(((1 << 20) + p.per_group - 1) / p.per_group);  // (exact for e < 1024)
  // 32 experts in question; a place for each expert where groups do not end with lanes
  p.slots = groups > 1 && p.group_shift < 0 && num_experts > 32 ? (int)num_experts : 32;
  const bool even = num_experts % 32 == 0 && (p.per & (p.per - 1)) == 0;
  const int piece = p.per * size < 16 ? p.per * size : 16;
  p.vector = even && aligned(logits, piece) && p.pitch % piece == 0 &&
             (!bias || aligned(bias, p.per * 4 < 16 ? p.per * 4 : 16));
  return p.per <= 1    ? launch<1>(p, stream)
         : p.per <= 2  ? launch<2>(p, stream)
         : p.per <= 4  ? launch<4>(p, stream)
         : p.per <= 8  ? launch<8>(p, stream)
         : p.per <= 16 ? launch<16>(p, stream)
                       : launch<32>(p, stream);
}
