// combine_experts.cu — combine_experts: each token's rows of the experts' last
// product, weighted and added up.
//
//   out[t] = base[t] + sum_j weights[t][j] * y[places[t][j]]
//
// Bound by memory: top_k rows read and one written for each token. A thread takes 32
// bytes of a row (16 where rows are aligned no better) and has the loads of up to 8
// rows in flight; the sum runs over j in order, in binary32. A block is one warp: 5003
// tokens x 8 rows of 7168 take 100 us, 6430 GB/s, and 104 with two warps; 16 bytes a
// thread and eight warps, which all go on at once to the same few rows, took 113. (Without
// a base a kernel of its own: 90 registers, 104 with one, and 105 us.)
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "kvq_device.cuh"
#include "kvq_experts.h"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kFlight = 8;

struct CombineParams {
  const uint8_t* y;
  const int64_t* places;
  const float* weights;
  const uint8_t* base;  // or null
  uint8_t* out;
  int64_t y_pitch, base_pitch, out_pitch;  // bytes
  int64_t num_rows;
  int top_k, vectors;
};

template <bool kHalf>
__device__ __forceinline__ void widen(uint32_t u, float& lo, float& hi) {
  if (kHalf) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u));
    lo = v.x;
    hi = v.y;
  } else {
    lo = bf16_lo(u);
    hi = bf16_hi(u);
  }
}

// kWords words of 32 bits.
template <int kWords>
struct Words {
  uint32_t u[kWords];
};
__device__ __forceinline__ void load(const uint8_t* p, Words<8>& v) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]), "=r"(v.u[4]), "=r"(v.u[5]),
                 "=r"(v.u[6]), "=r"(v.u[7])
               : "l"(p));
}
__device__ __forceinline__ void load(const uint8_t* p, Words<4>& v) {
  const uint4 w = ld_once_v4(p);
  v.u[0] = w.x;
  v.u[1] = w.y;
  v.u[2] = w.z;
  v.u[3] = w.w;
}
__device__ __forceinline__ void store(uint8_t* p, const Words<8>& v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.u[0]),
               "r"(v.u[1]), "r"(v.u[2]), "r"(v.u[3]), "r"(v.u[4]), "r"(v.u[5]), "r"(v.u[6]), "r"(v.u[7])
               : "memory");
}
__device__ __forceinline__ void store(uint8_t* p, const Words<4>& v) {
  st_v4(p, make_uint4(v.u[0], v.u[1], v.u[2], v.u[3]));
}

template <bool kHalf>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  uint32_t d;
  if (kHalf)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <bool kHalf, int kWords, bool kBase>
__global__ void __launch_bounds__(64) combine_experts_kernel(const CombineParams p) {
  const int64_t t = blockIdx.x;
  const int v = blockIdx.y * blockDim.x + threadIdx.x;
  if (v >= p.vectors) return;
  const int64_t at = 4 * kWords * (int64_t)v;
  const int64_t* places = p.places + t * p.top_k;
  const float* weights = p.weights + t * p.top_k;
  float acc[2 * kWords];
#pragma unroll
  for (int k = 0; k < 2 * kWords; ++k) acc[k] = 0.0f;
  uint4 base[kWords / 4];
  if (kBase) {  // (ordinary loads: out may be base)
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      base[i] = *reinterpret_cast<const uint4*>(p.base + t * p.base_pitch + at + 16 * i);
  }
  for (int j0 = 0; j0 < p.top_k; j0 += kFlight) {
    Words<kWords> x[kFlight];
    float w[kFlight];
    bool in[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      in[i] = false;
      if (j0 + i < p.top_k) {
        const int64_t place = __ldg(reinterpret_cast<const long long*>(places) + j0 + i);
        in[i] = place >= 0 && place < p.num_rows;
        w[i] = ld_f32(weights + j0 + i);
        if (in[i]) load(p.y + place * p.y_pitch + at, x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
      if (in[i]) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          float lo, hi;
          widen<kHalf>(x[i].u[k], lo, hi);
          acc[2 * k] = fmaf(w[i], lo, acc[2 * k]);
          acc[2 * k + 1] = fmaf(w[i], hi, acc[2 * k + 1]);
        }
      }
  }
  if (kBase) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint4 b = base[k / 4];
      float lo, hi;
      widen<kHalf>(k % 4 == 0 ? b.x : k % 4 == 1 ? b.y : k % 4 == 2 ? b.z : b.w, lo, hi);
      acc[2 * k] += lo;
      acc[2 * k + 1] += hi;
    }
  }
  Words<kWords> sum;
#pragma unroll
  for (int k = 0; k < kWords; ++k) sum.u[k] = narrow2<kHalf>(acc[2 * k], acc[2 * k + 1]);
  store(p.out + t * p.out_pitch + at, sum);
}

}  // namespace
}  // namespace kvq

extern "C" int combine_experts(const void* y, int64_t y_stride, int64_t num_rows,
                               const int64_t* places, const float* weights, int64_t num_tokens,
                               int64_t top_k, const void* base, int64_t base_stride, void* out,
                               int64_t out_stride, int64_t n, int32_t dtype, cudaStream_t stream) {
  using namespace kvq;
  if (num_tokens < 0 || num_tokens > 0x7FFFFFFF || num_rows < 0 || num_rows > 0x7FFFFFFF)
    return KVQ_EINVAL;
  if ((dtype != KVQ_BF16 && dtype != KVQ_FP16) || top_k < 1 || top_k > 32) return KVQ_EINVAL;
  if (n < 8 || n > (1 << 24) || n % 8) return KVQ_EINVAL;
  const auto bad = [](int64_t s, int64_t least) { return s < least || s % 8 || s > (1ll << 30); };
  if (bad(y_stride, 0) || bad(out_stride, n) || (base && bad(base_stride, 0))) return KVQ_EINVAL;
  if (num_tokens == 0) return KVQ_OK;
  if ((!y && num_rows) || !places || !weights || !out || !aligned(y, 16) || !aligned(places, 8) ||
      !aligned(weights, 4) || !aligned(base, 16) || !aligned(out, 16))
    return KVQ_EINVAL;
  if (base == out && base_stride != out_stride) return KVQ_EINVAL;
  CombineParams p;
  p.y = static_cast<const uint8_t*>(y);
  p.places = places;
  p.weights = weights;
  p.base = static_cast<const uint8_t*>(base);
  p.out = static_cast<uint8_t*>(out);
  p.y_pitch = y_stride * 2;
  p.base_pitch = base_stride * 2;
  p.out_pitch = out_stride * 2;
  p.num_rows = num_rows;
  p.top_k = (int)top_k;
  const bool wide = n % 16 == 0 && aligned(y, 32) && aligned(out, 32) && p.y_pitch % 32 == 0 &&
                    p.out_pitch % 32 == 0;
  p.vectors = (int)(n / (wide ? 16 : 8));
  const unsigned threads = wide ? 32 : 64;  // (the grid has at most 65535 blocks of columns)
  const dim3 grid((unsigned)num_tokens, (p.vectors + threads - 1) / threads);
  const auto launch = [&](auto half, auto base_too) {
    if (wide)
      combine_experts_kernel<half(), 8, base_too()><<<grid, threads, 0, stream>>>(p);
    else
      combine_experts_kernel<half(), 4, base_too()><<<grid, threads, 0, stream>>>(p);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (dtype == KVQ_FP16)
    base ? launch(Yes{}, Yes{}) : launch(Yes{}, No{});
  else
    base ? launch(No{}, Yes{}) : launch(No{}, No{});
  return launch_status();
}
