// combine_experts.cu — combine_experts: each token's rows of the experts' last
// product, weighted and added up.
//
//   out[t] = base[t] + sum_j weights[t][j] * y[places[t][j]]
//
// Bound by memory: top_k rows read and one written for each token. A thread
// takes 8 neighbouring values; the loads of up to 8 rows are in flight at once.
// The sum runs over j in order, in binary32.
#include <cuda_fp16.h>

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_experts.h"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;
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
__device__ __forceinline__ void widen(uint4 w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kHalf) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    } else {
      f[2 * i] = bf16_lo(u[i]);
      f[2 * i + 1] = bf16_hi(u[i]);
    }
  }
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

template <bool kHalf>
__global__ void __launch_bounds__(kThreads) combine_experts_kernel(const CombineParams p) {
  const int64_t t = blockIdx.x;
  const int v = blockIdx.y * kThreads + threadIdx.x;
  if (v >= p.vectors) return;
  const int64_t* places = p.places + t * p.top_k;
  const float* weights = p.weights + t * p.top_k;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  uint4 base = make_uint4(0, 0, 0, 0);
  if (p.base)  // (an ordinary load: out may be base)
    base = *reinterpret_cast<const uint4*>(p.base + t * p.base_pitch + 16 * (int64_t)v);
  for (int j0 = 0; j0 < p.top_k; j0 += kFlight) {
    uint4 x[kFlight];
    float w[kFlight];
    bool in[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      in[i] = false;
      if (j0 + i < p.top_k) {
        const int64_t place = __ldg(reinterpret_cast<const long long*>(places) + j0 + i);
        in[i] = place >= 0 && place < p.num_rows;
        w[i] = ld_f32(weights + j0 + i);
        if (in[i]) x[i] = ld_once_v4(p.y + place * p.y_pitch + 16 * (int64_t)v);
      }
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
      if (in[i]) {
        float f[8];
        widen<kHalf>(x[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[i], f[k], acc[k]);
      }
  }
  if (p.base) {
    float f[8];
    widen<kHalf>(base, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += f[k];
  }
  st_v4(p.out + t * p.out_pitch + 16 * (int64_t)v,
        make_uint4(narrow2<kHalf>(acc[0], acc[1]), narrow2<kHalf>(acc[2], acc[3]),
                   narrow2<kHalf>(acc[4], acc[5]), narrow2<kHalf>(acc[6], acc[7])));
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
  p.vectors = (int)(n / 8);
  const int threads = p.vectors < kThreads ? (p.vectors + 31) / 32 * 32 : kThreads;
  const dim3 grid((unsigned)num_tokens, (unsigned)((p.vectors + kThreads - 1) / kThreads));
  if (dtype == KVQ_FP16)
    combine_experts_kernel<true><<<grid, threads, 0, stream>>>(p);
  else
    combine_experts_kernel<false><<<grid, threads, 0, stream>>>(p);
  return launch_status();
}
