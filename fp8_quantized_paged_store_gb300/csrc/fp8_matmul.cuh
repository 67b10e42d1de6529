// fp8_matmul.cuh — what the two kernels of the block-scaled 8-bit products
// share: parameters, the tiles of the experts' rows, PTX for 8-bit operands,
// and the write of a gated result.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "kvq_device.cuh"
#include "tcgen05.cuh"

namespace kvq {

constexpr int kGroupK = 128;       // values of a scale group: one step of a tile
constexpr int kMaxExperts = 1024;

struct MatmulParams {
  CUtensorMap a_map, b_map, out_map;
  const uint8_t* a;
  const float* a_scales;
  const float* b_scales;
  const int64_t* offsets;  // null: one matrix
  const int64_t* rows;     // null: row i itself
  uint8_t* out;
  float* out_scales;  // gated
  int32_t* status;
  int64_t a_stride, k;
  int64_t a_scale_stride, b_scale_stride, b_scale_expert_stride;  // floats
  int64_t out_pitch;                                              // bytes
  int64_t out_scale_stride;                                       // floats
  int a_rows, num_rows, experts;  // experts >= 1
  int n;                          // columns of the result
  int steps;                      // groups of k
  int a_group_step;               // 0: one scale for a whole row
  int row_tiles_dense;            // tiles of rows without experts
  int column_tiles;
  int half;       // fp16 result
  int up_blocks;  // gated: blocks of 128 weights' rows from gate to up
  int blocks;     // of 128 weights' rows
  int wide;       // out's rows are 16-byte aligned (2: 32-byte)
};

// First tile and first row of every expert, in shared memory.
struct ExpertTiles {
  int tile_start[kMaxExperts + 1];
  int row_start[kMaxExperts + 1];
  int warp_sums[32];

  __device__ __forceinline__ int rows(int e) const {
    const int n = row_start[e + 1] - row_start[e];
    return n > 0 ? n : 0;
  }
};

__device__ __forceinline__ int clamp_row(int64_t v, int rows) {
  return v < 0 ? 0 : v > rows ? rows : (int)v;
}

// Counts the tiles of kRows rows x one block of columns of every expert; called
// by the whole block of kThreads.
template <int kRows, int kThreads>
__device__ __forceinline__ void count_tiles(const MatmulParams& p, ExpertTiles& s) {
  const int tid = threadIdx.x;
  if (!p.offsets) {
    if (tid == 0) {
      s.tile_start[0] = 0;
      s.tile_start[1] = p.row_tiles_dense * p.column_tiles;
      s.row_start[0] = 0;
      s.row_start[1] = p.num_rows;
    }
    __syncthreads();
    return;
  }
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  const int per = (p.experts + kThreads - 1) / kThreads;
  int sum = 0, mine[kPer];
  bool falling = false;  // (then no expert has rows: tiles would overlap, and be more than the grid's)
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    mine[i] = 0;
    const int e = tid * per + i;
    if (i < per && e < p.experts) {
      const int low = clamp_row(p.offsets[e], p.num_rows);
      const int high = clamp_row(p.offsets[e + 1], p.num_rows);
      const int rows = high > low ? high - low : 0;
      falling = falling || high < low;
      s.row_start[e] = low;
      if (e == p.experts - 1) s.row_start[p.experts] = high;
      mine[i] = (rows + kRows - 1) / kRows * p.column_tiles;
      sum += mine[i];
    }
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if ((tid & 31) >= o) upto += v;
  }
  if ((tid & 31) == 31) s.warp_sums[tid >> 5] = upto;
  falling = __syncthreads_or(falling);
  int before = upto - sum;
  for (int w = 0; w < (tid >> 5); ++w) before += s.warp_sums[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * per + i;
    if (i < per && e < p.experts) {
      s.tile_start[e] = before;
      before += mine[i];
      if (e == p.experts - 1) s.tile_start[p.experts] = falling ? 0 : before;
    }
  }
  __syncthreads();
}

// The expert that the index-th tile belongs to.
__device__ __forceinline__ int expert_of_tile(const MatmulParams& p, const ExpertTiles& s,
                                              int index) {
  int low = 0, high = p.experts;
  while (high - low > 1) {
    const int mid = (low + high) >> 1;
    if (s.tile_start[mid] <= index)
      low = mid;
    else
      high = mid;
  }
  return low;
}

// ------------------------------------------------------------- tensor cores ---

// As mma_ss with E4M3 operands: 32 values of K.
__device__ __forceinline__ void mma_ss_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, E4M3 operands, both
// K-major.
__host__ __device__ constexpr uint32_t instr_desc_f8(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One box of a 2-D tensor map.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// Four rows of a 2-D tensor map whose box is one row.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int y0,
                                            int y1, int y2, int y3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(bar)
      : "memory");
}

// One lane of a converged warp; the compiler knows that it is one, so that what it
// issues takes its operands from uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Bounded waits of a converged warp, which stay converged: every branch goes by a
// vote, so that the compiler takes what follows for uniform. (In code that it takes for
// divergent, sums in registers ran at half their rate.)
__device__ __forceinline__ bool gone(uint32_t abort) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(abort) : "memory");
  return __any_sync(0xFFFFFFFFu, v != 0);
}
__device__ __forceinline__ void give_up(uint32_t abort) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1) : "memory");
}
__device__ __forceinline__ bool uniform_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity))) return true;
    if ((i & 31u) == 31u && gone(abort)) return false;
  }
  give_up(abort);
  return false;
}
// For both barriers' phases, tested together: a test takes 57 cycles of a waiting
// warp, whether the phase is complete or not.
__device__ __forceinline__ bool uniform_wait2(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb,
                                              uint32_t abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    const bool da = mbar_test(a, pa), db = mbar_test(b, pb);
    if (__all_sync(0xFFFFFFFFu, da && db)) return true;
    if ((i & 31u) == 31u && gone(abort)) return false;
  }
  give_up(abort);
  return false;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Row i's place in a, clamped into it; `ok`: it lies there.
__device__ __forceinline__ int a_row(const MatmulParams& p, int i, bool& ok) {
  if (!p.rows) {
    ok = i < p.a_rows;
    return ok ? i : p.a_rows - 1;
  }
  const int64_t r = p.rows[i];
  ok = r >= 0 && r < p.a_rows;
  return ok ? (int)r : 0;
}

// ----------------------------------------------------------------- clusters ---

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cluster(uint32_t a, uint32_t rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
  return d;
}
// A store to a block's shared memory, another one's or the own, that counts towards a
// barrier there.
__device__ __forceinline__ void st_async4(uint32_t a, const float* v, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(bar)
      : "memory");
}
// The cluster's own barrier in two parts, where no data passes with it.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_all() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// uniform_wait for data of other blocks of the cluster. (Waits and arrivals of cluster
// scope cost about 1000 cycles: only where data of shared memory passes.)
__device__ __forceinline__ bool cluster_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(0xFFFFFFFFu, done != 0)) return true;
    if ((i & 31u) == 31u && gone(abort)) return false;
  }
  give_up(abort);
  return false;
}

// ---------------------------------------------------------------- results ---

__device__ __forceinline__ uint32_t narrow2_to(float lo, float hi, bool half) {
  uint32_t d;
  if (half)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// silu(gate) * up. The exponential and the reciprocal are the device's fast ones. By their
// documented errors, 2 + 1.173 |gate| and 1 units in the last place (2^-23), and a rounding,
// 2^-24, each of 1 + exp and of the two products, it is within (9 + 2.35 |gate|) 2^-24 of the
// value, relative to it: 2^-18.4 for |gate| = 16, 2^-17 for 50 (the result's codes have 4
// bits, its scale 24). 0 where exp(-gate) overflows.
__device__ __forceinline__ float gated(float gate, float up) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-gate)));
  return gate * r * up;
}

// A group's scale and the factor from values to codes, of its largest |z|
// (the floor first, as add_rmsnorm_fp8 does). z times the factor is within 3 roundings,
// 2^-22, of z / scale.
__device__ __forceinline__ float code_scale(float top) { return fmaxf(top, 1e-4f) / 448.0f; }
__device__ __forceinline__ float code_factor(float top) {
  return top >= 1e-4f ? 448.0f / top : 1.0f / (1e-4f / 448.0f);
}

int launch_matmul_tiles(const MatmulParams& p, bool is_gated, cudaStream_t stream);
int launch_matmul_few(const MatmulParams& p, bool is_gated, int row_tile, cudaStream_t stream);

}  // namespace kvq
