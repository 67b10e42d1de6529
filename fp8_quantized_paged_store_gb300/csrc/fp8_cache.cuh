// fp8_cache.cuh — what the kernels on the paged E4M3 cache share: its
// addressing, the ragged sequences, and block-wide searches over them.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_fp8.h"
#include "kvq_host.h"

namespace kvq {

struct Fp8Cache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int64_t num_pages;
  int64_t page_stride, head_stride;  // bytes
  int64_t scale_page_stride;
  const int64_t* table;
  int64_t table_stride;
  int64_t capacity;  // max_pages * page_size: tokens a sequence can have
  int32_t slot_stride;
  int32_t page_log2;
};

struct Fp8Seqs {
  const int64_t* start;  // [count + 1]
  const int64_t* lens;   // context_lens or seq_lens, [count]
  int64_t num_tokens;
  int32_t count;
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// First row and number of rows of sequence s, within [0, num_tokens].
__device__ __forceinline__ void seq_rows(const Fp8Seqs& q, int s, int64_t& first, int64_t& n) {
  first = clamp64(q.start[s], 0, q.num_tokens);
  const int64_t end = clamp64(q.start[s + 1], 0, q.num_tokens);
  n = end > first ? end - first : 0;
}

// Page that holds a token of sequence s, or -1 when the table names none.
__device__ __forceinline__ int64_t page_of(const Fp8Cache& c, int64_t s, int64_t token) {
  const int64_t g = c.table[s * c.table_stride + (token >> c.page_log2)];
  return (uint64_t)g < (uint64_t)c.num_pages ? g : -1;
}

// Finds the sequence whose share of a running total contains a place in it:
// weight(s) >= 0 is sequence s's share, place(total) the place wanted, and on
// return s is the sequence with total(0..s-1) <= place < total(0..s) and
// `before` the former. False when the place lies past the total. Called by a
// whole block of kThreads threads; thread i adds up the shares of one run of
// sequences, so every share is worked out once, all of them in parallel.
template <int kThreads, typename T, typename Weight, typename Place>
__device__ __forceinline__ bool find_share(int count, Weight weight, Place place, int& s,
                                           T& before, T& total) {
  __shared__ T warp_sums[kThreads / 32];
  __shared__ T found_before;
  __shared__ int found_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (count + kThreads - 1) / kThreads;
  const int first = threadIdx.x * per, last = min(first + per, count);
  T mine = 0;
#pragma unroll 1
  for (int i = first; i < last; ++i) mine += weight(i);
  T scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) warp_sums[warp] = scan;
  __syncthreads();
  T base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const T x = warp_sums[w];
    if (w < warp) base += x;
    total += x;
  }
  const T at = place(total);
  if (at >= total) return false;  // the same for all threads
  T upto = base + scan - mine;
  if (at >= upto && at < upto + mine) {
#pragma unroll 1
    for (int i = first; i < last; ++i) {
      const T x = per == 1 ? mine : weight(i);
      if (at < upto + x) {
        found_s = i;
        found_before = upto;
        break;
      }
      upto += x;
    }
  }
  __syncthreads();
  s = found_s;
  before = found_before;
  return true;
}

// ------------------------------------------------------------- E4M3, fp16 ---

// Four E4M3 codes as two pairs of fp16 values, exactly; code 0x7F is NaN.
// (The halves of the word are named as 16-bit registers: shifting the upper
// one down first cost an instruction more for each pair.)
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two values of the row type (bf16 or fp16) as binary32, and back.
__device__ __forceinline__ float2 widen2(uint32_t w, bool half) {
  return half ? f16x2_to_f32(w) : make_float2(bf16_lo(w), bf16_hi(w));
}

__device__ __forceinline__ uint32_t narrow2(float lo, float hi, bool half) {
  uint32_t d;
  if (half)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ void widen8(uint4 w, bool half, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = widen2(u[i], half);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8], bool half) {
  return make_uint4(narrow2(f[0], f[1], half), narrow2(f[2], f[3], half),
                    narrow2(f[4], f[5], half), narrow2(f[6], f[7], half));
}

// ------------------------------------------------------------ host checks ---

// Whether runs of `extent`, one for every place in dimensions of these sizes and
// strides, lie apart: each stride, the smallest first, passes all that the
// dimensions below it span.
template <int kDims>
inline bool runs_apart(int64_t extent, const int64_t (&size)[kDims],
                       const int64_t (&stride)[kDims]) {
  bool done[kDims] = {};
  for (int n = 0; n < kDims; ++n) {
    int next = -1;
    for (int i = 0; i < kDims; ++i)
      if (!done[i] && (next < 0 || stride[i] < stride[next])) next = i;
    done[next] = true;
    if (size[next] < 2) continue;
    if (stride[next] < extent) return false;
    extent += (size[next] - 1) * stride[next];
  }
  return true;
}

// Checks shared by the entry points on the cache; fills `c`. A row of the block
// table may stand for all sequences (stride 0), and where the cache is only
// read one page's scales for all pages.
inline bool fp8_cache_params(uint8_t* k_cache, uint8_t* v_cache, int64_t num_pages,
                             int64_t page_size, int64_t page_stride, int64_t head_stride,
                             int64_t slot_stride, uint8_t* k_scales, uint8_t* v_scales,
                             int64_t scale_page_stride, const int64_t* block_table,
                             int64_t table_stride, int64_t max_pages, int64_t num_seqs,
                             int64_t num_kv_heads, int64_t head_dim, bool written, Fp8Cache& c) {
  if (num_pages < 1 || num_pages > (int64_t)1 << 40) return false;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return false;
  if (num_kv_heads < 1 || num_kv_heads > 65535) return false;
  if (max_pages < 0 || max_pages > (int64_t)1 << 32) return false;
  if (table_stride < max_pages && table_stride != 0) return false;
  if (table_stride > INT64_MAX / 16 / (num_seqs + 1)) return false;
  const int64_t cap = INT64_MAX / 4;
  if (slot_stride < head_dim || slot_stride > (int64_t)1 << 22 || slot_stride % 16) return false;
  if (head_stride < 0 || head_stride % 16 || head_stride > cap / num_kv_heads) return false;
  if (page_stride < 0 || page_stride % 16 || page_stride > cap / num_pages) return false;
  if (scale_page_stride < num_kv_heads && (written || scale_page_stride != 0)) return false;
  if (scale_page_stride > cap / num_pages) return false;
  if (written && !runs_apart<3>(head_dim, {num_pages, num_kv_heads, page_size},
                                {page_stride, head_stride, slot_stride}))
    return false;
  c.k = k_cache;
  c.v = v_cache;
  c.k_scales = k_scales;
  c.v_scales = v_scales;
  c.num_pages = num_pages;
  c.page_stride = page_stride;
  c.head_stride = head_stride;
  c.scale_page_stride = scale_page_stride;
  c.table = block_table;
  c.table_stride = table_stride;
  c.capacity = max_pages * page_size;
  c.slot_stride = (int32_t)slot_stride;
  c.page_log2 = __builtin_ctzll((unsigned long long)page_size);
  return true;
}

}  // namespace kvq
