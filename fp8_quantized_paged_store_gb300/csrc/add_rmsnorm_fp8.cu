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
// byte is read once. Above the floor y / scale is 448 u / max |u| for any
// multiple u of y: with u = h * w times a power of two, the sum's and the
// root's roundings stay out of the codes: u, max |u|, their quotient's factor
// and the product round once each (u twice with a residual). A group of 128 is
// 16 neighbouring threads (vector v of a thread is thread + v * blockDim), so
// its maximum needs four shuffles and no barrier.
//
// Many tokens take four vectors a thread (64 bytes of each input in flight, a
// quarter of the warps at each barrier), few tokens one (a token's chain is
// shorter): 8192 x 7168 with residual and groups 67 us (6150 GB/s) against 87,
// 5003 x 5120 without residual 17.6 us against 25; at 456 tokens of 7168 4.3
// us against 5.2, up to two tokens an SM the same or better with one.
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

// Sum over the block; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* slots) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? slots[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Largest of values >= +0 over the block: their bits are ordered as they are.
__device__ __forceinline__ float block_max(float v, uint32_t* slots) {
  uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slots[threadIdx.x >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? slots[lane] : 0u);
  return __uint_as_float(m);
}

template <int kVec, bool kGroups, bool kHalf, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) add_rmsnorm_fp8_kernel(const NormParams p) {
  __shared__ float sums[32];
  __shared__ uint32_t tops[32];
  const int64_t t = blockIdx.x;
  const uint8_t* xr = p.x + t * p.x_pitch;
  float h[kVec][8];
  float sum = 0.0f;
  {
    uint4 xv[kVec], rv[kVec];
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
      widen(xv[i], kHalf, h[i]);
      if (p.residual) {
        float r[8];
        widen(rv[i], kHalf, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] += r[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(h[i][k], h[i][k], sum);
      const int v = threadIdx.x + i * blockDim.x;
      if (p.residual_out && v < p.vectors)
        st_v4(p.residual_out + t * p.residual_out_pitch + 16 * v,
              make_uint4(narrow2(h[i][0], h[i][1], kHalf), narrow2(h[i][2], h[i][3], kHalf),
                         narrow2(h[i][4], h[i][5], kHalf), narrow2(h[i][6], h[i][7], kHalf)));
    }
  }
  uint4 wv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    wv[i] = v < p.vectors ? ld_nc_v4(p.weight + 16 * v) : make_uint4(0, 0, 0, 0);
  }
  sum = block_sum(sum, sums);
  // 1 / rms as a power of two and a factor in [1, 2)
  const float r = 1.0f / sqrtf(sum * p.hidden_inv + p.eps);
  const bool split = r >= 1.1754944e-38f && r <= 3.4028235e38f;  // not 0, infinite or NaN
  const float r_pow = split ? __uint_as_float(__float_as_uint(r) & 0x7F800000u) : r;
  const float r_rest =
      split ? __uint_as_float((__float_as_uint(r) & 0x007FFFFFu) | 0x3F800000u) : 1.0f;
  float amax[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    float w[8];
    widen(wv[i], kHalf, w);
    amax[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[i][k] = h[i][k] * r_pow * w[k];
      amax[i] = fmaxf(amax[i], fabsf(h[i][k]));
    }
    if (kGroups) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xFFFFFFFFu, amax[i], o));
    }
  }
  float to[kVec];
  if (kGroups) {
    // 16 threads share each of their kVec groups: thread i of them works out
    // the i-th one's scale
    const int own = threadIdx.x & 15;
    float top = amax[0];
#pragma unroll
    for (int i = 1; i < kVec; ++i) top = own == i ? amax[i] : top;
    const float scale = fmaxf(top * r_rest, 1e-4f) / 448.0f;
    const float to_code = top * r_rest >= 1e-4f ? 448.0f / top : r_rest / (1e-4f / 448.0f);
    const int group = (int)(threadIdx.x + own * blockDim.x) >> 4;
    if (own < kVec && 16 * group < p.vectors) p.scales[t * p.scale_stride + group] = scale;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      to[i] = __shfl_sync(0xFFFFFFFFu, to_code, (int)(threadIdx.x & 16) + i);
  } else {
#pragma unroll
    for (int i = 1; i < kVec; ++i) amax[0] = fmaxf(amax[0], amax[i]);
    const float top = block_max(amax[0], tops);
    if (threadIdx.x == 0) p.scales[t * p.scale_stride] = fmaxf(top * r_rest, 1e-4f) / 448.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      to[i] = top * r_rest >= 1e-4f ? 448.0f / top : r_rest / (1e-4f / 448.0f);
  }
  uint8_t* orow = p.out + t * p.out_pitch;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= p.vectors) continue;
    st_v2(orow + 8 * v,
          cvt_e4m3x2(h[i][0] * to[i], h[i][1] * to[i]) |
              (cvt_e4m3x2(h[i][2] * to[i], h[i][3] * to[i]) << 16),
          cvt_e4m3x2(h[i][4] * to[i], h[i][5] * to[i]) |
              (cvt_e4m3x2(h[i][6] * to[i], h[i][7] * to[i]) << 16));
  }
}

template <int kVec, int kThreads, int kBlocks>
void launch(const NormParams& p, bool groups, bool half, unsigned tokens, cudaStream_t stream) {
  const int n = (p.vectors + kVec - 1) / kVec;
  auto* kernel = groups ? (half ? add_rmsnorm_fp8_kernel<kVec, true, true, kThreads, kBlocks>
                                : add_rmsnorm_fp8_kernel<kVec, true, false, kThreads, kBlocks>)
                        : (half ? add_rmsnorm_fp8_kernel<kVec, false, true, kThreads, kBlocks>
                                : add_rmsnorm_fp8_kernel<kVec, false, false, kThreads, kBlocks>);
  kernel<<<tokens, (n + 31) / 32 * 32, 0, stream>>>(p);
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
  const unsigned tokens = (unsigned)num_tokens;
  const bool half = dtype == KVQ_FP16;
  if (p.vectors > 1024)
    launch<4, 1024, 1>(p, group != 0, half, tokens, stream);
  else if (num_tokens > 2 * sm_count())
    launch<4, 256, 4>(p, group != 0, half, tokens, stream);
  else
    launch<1, 1024, 1>(p, group != 0, half, tokens, stream);
  return launch_status();
}
