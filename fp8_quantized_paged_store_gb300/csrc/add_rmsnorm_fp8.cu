// add_rmsnorm_fp8.cu — add_rmsnorm_fp8: h = x + residual, RMSNorm of h with a
// weight, and the result as E4M3 codes with one binary32 scale for each token
// or each 128 values.
//
//   r = 1 / sqrt(sum(h^2) / H + eps),  y = h * r * w,
//   scale = max(max |y| over the group, 1e-4) / 448,  code = E4M3(y / scale)
//
// Bound by memory: 2 + 2 bytes read and 2 + 1 written per element. One block
// takes a token; its row stays in registers (kVec vectors of 8 values a
// thread) between the sum, the group's maximum and the codes, so every input
// byte is read once. A group of 128 is 16 neighbouring threads (vector v of a
// thread is thread + v * blockDim), so its maximum needs four shuffles and no
// barrier.
#include <cuda_fp16.h>

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_fp8.h"
#include "kvq_host.h"

namespace kvq {
namespace {

struct NormParams {
  const uint8_t* x;
  const uint8_t* residual;  // or null
  const uint8_t* weight;
  uint8_t* out;
  float* scales;
  uint8_t* residual_out;  // or null
  int64_t x_pitch, residual_pitch, residual_out_pitch;  // bytes
  int64_t out_pitch;                                    // bytes
  int64_t scale_stride;                                 // floats
  float eps, hidden_inv;
  int vectors;  // hidden / 8
  int half;     // 1: fp16, 0: bf16
};

__device__ __forceinline__ void widen(uint4 w, bool half, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (half) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    } else {
      f[2 * i] = bf16_lo(u[i]);
      f[2 * i + 1] = bf16_hi(u[i]);
    }
  }
}

__device__ __forceinline__ uint32_t narrow2(float lo, float hi, bool half) {
  uint32_t d;
  if (half)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 16 bytes of a row that this kernel may also write (residual_out in place):
// an ordinary load, not one through the read-only path.
__device__ __forceinline__ uint4 ld_row(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Sum (or maximum) over the block; every thread gets it. The two uses in the
// kernel take different slots, so neither waits for the other's readers.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* slots) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  return v;
}

template <int kVec, bool kGroups>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(const NormParams p) {
  __shared__ float slots[64];
  const int64_t t = blockIdx.x;
  const uint8_t* xr = p.x + t * p.x_pitch;
  const bool half = p.half != 0;
  uint4 xv[kVec], rv[kVec], wv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    xv[i] = v < p.vectors ? ld_row(xr + 16 * v) : make_uint4(0, 0, 0, 0);
  }
  if (p.residual) {
    const uint8_t* rr = p.residual + t * p.residual_pitch;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      rv[i] = v < p.vectors ? ld_row(rr + 16 * v) : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    wv[i] = v < p.vectors ? ld_nc_v4(p.weight + 16 * v) : make_uint4(0, 0, 0, 0);
  }
  float h[kVec][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    widen(xv[i], half, h[i]);
    if (p.residual) {
      float r[8];
      widen(rv[i], half, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] += r[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(h[i][k], h[i][k], sum);
    const int v = threadIdx.x + i * blockDim.x;
    if (p.residual_out && v < p.vectors)
      st_v4(p.residual_out + t * p.residual_out_pitch + 16 * v,
            make_uint4(narrow2(h[i][0], h[i][1], half), narrow2(h[i][2], h[i][3], half),
                       narrow2(h[i][4], h[i][5], half), narrow2(h[i][6], h[i][7], half)));
  }
  sum = block_reduce<false>(sum, slots);
  const float r = 1.0f / sqrtf(sum * p.hidden_inv + p.eps);
  float amax[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    float w[8];
    widen(wv[i], half, w);
    amax[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[i][k] = h[i][k] * r * w[k];
      amax[i] = fmaxf(amax[i], fabsf(h[i][k]));
    }
    if (kGroups) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xFFFFFFFFu, amax[i], o));
    }
  }
  if (!kGroups) {
#pragma unroll
    for (int i = 1; i < kVec; ++i) amax[0] = fmaxf(amax[0], amax[i]);
    const float m = block_reduce<true>(amax[0], slots + 32);
#pragma unroll
    for (int i = 0; i < kVec; ++i) amax[i] = m;
    if (threadIdx.x == 0) p.scales[t * p.scale_stride] = fmaxf(m, 1e-4f) / 448.0f;
  }
  uint8_t* orow = p.out + t * p.out_pitch;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= p.vectors) continue;
    const float scale = fmaxf(amax[i], 1e-4f) / 448.0f;
    const float inv = 1.0f / scale;
    if (kGroups && (threadIdx.x & 15) == 0) p.scales[t * p.scale_stride + (v >> 4)] = scale;
    st_v2(orow + 8 * v,
          cvt_e4m3x2(h[i][0] * inv, h[i][1] * inv) | (cvt_e4m3x2(h[i][2] * inv, h[i][3] * inv) << 16),
          cvt_e4m3x2(h[i][4] * inv, h[i][5] * inv) | (cvt_e4m3x2(h[i][6] * inv, h[i][7] * inv) << 16));
  }
}

}  // namespace
}  // namespace kvq

extern "C" int add_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual,
                               int64_t residual_stride, const void* weight, float eps,
                               int32_t dtype, int64_t num_tokens, int64_t hidden, int32_t group,
                               uint8_t* out, int64_t out_stride, float* scales,
                               int64_t scale_stride, void* residual_out,
                               int64_t residual_out_stride, cudaStream_t stream) {
  using namespace kvq;
  if (num_tokens < 0 || num_tokens > 0x7FFFFFFF || (dtype != KVQ_BF16 && dtype != KVQ_FP16))
    return KVQ_EINVAL;
  if (hidden < 8 || hidden > 32768 || hidden % 8 || (group != 0 && group != 128)) return KVQ_EINVAL;
  if (group && hidden % group) return KVQ_EINVAL;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return KVQ_EINVAL;
  const int64_t cap = INT64_MAX / 8 / (num_tokens + 1);
  auto bad = [&](int64_t s, int64_t least, int64_t unit) {
    return s < least || s % unit || s > cap;
  };
  if (bad(x_stride, hidden, 8) || bad(out_stride, hidden, 8) ||
      bad(scale_stride, group ? hidden / group : 1, 1))
    return KVQ_EINVAL;
  if (residual && bad(residual_stride, hidden, 8)) return KVQ_EINVAL;
  if (residual_out && bad(residual_out_stride, hidden, 8)) return KVQ_EINVAL;
  if (num_tokens == 0) return KVQ_OK;
  if (!x || !weight || !out || !scales || (residual_out && !residual)) return KVQ_EINVAL;
  if ((residual_out == x && residual_out_stride != x_stride) ||
      (residual_out && residual_out == residual && residual_out_stride != residual_stride))
    return KVQ_EINVAL;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(out, 8) || !aligned(scales, 4) ||
      !aligned(residual, 16) || !aligned(residual_out, 16))
    return KVQ_EINVAL;
  NormParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.residual = static_cast<const uint8_t*>(residual);
  p.weight = static_cast<const uint8_t*>(weight);
  p.out = out;
  p.scales = scales;
  p.residual_out = static_cast<uint8_t*>(residual_out);
  p.x_pitch = x_stride * 2;
  p.residual_pitch = residual_stride * 2;
  p.residual_out_pitch = residual_out_stride * 2;
  p.out_pitch = out_stride;
  p.scale_stride = scale_stride;
  p.eps = eps;
  p.hidden_inv = 1.0f / (float)hidden;
  p.vectors = (int)(hidden / 8);
  p.half = dtype == KVQ_FP16;
  const unsigned grid = (unsigned)num_tokens;
  auto threads = [&](int vec) {
    const int n = (p.vectors + vec - 1) / vec;
    return (unsigned)((n + 31) / 32 * 32);
  };
  if (p.vectors <= 1024) {
    if (group)
      add_rmsnorm_fp8_kernel<1, true><<<grid, threads(1), 0, stream>>>(p);
    else
      add_rmsnorm_fp8_kernel<1, false><<<grid, threads(1), 0, stream>>>(p);
  } else {
    if (group)
      add_rmsnorm_fp8_kernel<4, true><<<grid, threads(4), 0, stream>>>(p);
    else
      add_rmsnorm_fp8_kernel<4, false><<<grid, threads(4), 0, stream>>>(p);
  }
  return launch_status();
}
