// fp8_matmul_few.cu — the kernel of the block-scaled 8-bit products for few
// rows to a matrix: decode batches, experts with few tokens.
//
//   out[i][j] = sum_g sa[i][g] sb[j/128][g] sum_{l in g} a[i][l] b[j][l]
//
// Bound by the weights' bytes. The product is taken the other way round: 128
// of b's rows are the M side of tcgen05.mma (kind::f8f6f4, E4M3 exact, fp32
// accumulators), up to 64 of a's rows its N side, so no tensor work is lost on
// rows that do not exist, and a block of 128 weights' rows has one scale for a
// group. One step is a group of 128 values: 16 KB of weights and kTok rows of 128
// bytes by TMA into 128-byte-swizzled stages, four MMAs into one of the
// accumulators in tensor memory, and, one feature to a thread,
//   acc[t] += partial[t] * (sa[t] sb)
// in registers. Roles: warps 0-3 (gated: 4-7 too, for the up half) add up and
// write, then one warp each for TMA, MMA issue and scales.
//
// Tiles are (expert, rows, block of columns), taken in turn by resident
// blocks; the loads run ahead over a tile's end. Few tiles are split over K among the
// blocks of a cluster: each rank owns some rows, and the others' sums of these come by
// asynchronous stores that count towards a barrier of the owner's shared memory (added in
// a fixed order).
//
// Measured: experts' weights of 462 MB in 72 us (6430 GB/s, 95 % of the copy bandwidth);
// one matrix of 6144 x 4096 by 8 rows in 8.9 us, of which 2 are the launch, 1 the first
// load's trip, 3 the steps, 1 the meeting of the sums and their way out.
#include "fp8_matmul.cuh"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kFactorSlots = 8;
// Blocks of a cluster, as many as fit and have a step: 8 x 1024 x 1024 takes 4.8 us by
// blocks of one step, 5.5 of four and 6.2 of eight, 64 x 512 x 1024 6.2, 7.6 and 8.2.
constexpr int kMostSplit = 8;
// Steps loaded before the block has started (more of them hold the start up).
constexpr int kEarly = 3;

template <int kTok, bool kGated>
struct Few {
  static constexpr int kHalves = kGated ? 2 : 1;
  static constexpr int kSumWarps = 4 * kHalves;
  static constexpr int kLoadWarp = kSumWarps, kMmaWarp = kSumWarps + 1, kScaleWarp = kSumWarps + 2;
  static constexpr int kThreads = 32 * (kSumWarps + 3);
  static constexpr uint32_t kWeightBytes = 128 * kGroupK;
  static constexpr uint32_t kStageBytes = kHalves * kWeightBytes + kTok * kGroupK;
  // Accumulators, and how many of them the sums take at a time: the waits of a step last
  // longer than the sums of 16 rows (256 ns a step one at a time; 8 x 4096 x 6144 went from
  // 9.6 to 8.9 us, 64 x 4096 x 4096, with the exchange in fours, from 12.4 to 10.3).
  static constexpr int kBatch = 64 / kTok;
  static constexpr int kBufs = kBatch > 2 ? 2 * kBatch : 4;
  static constexpr uint32_t kAccCols = kHalves * kTok;
  static constexpr uint32_t kTmemCols = kBufs * kAccCols < 32 ? 32 : kBufs * kAccCols;
  // exchange of the halves' or the cluster's sums: [rank of the sums][row of the owner's
  // / 4][feature][row % 4] (a split of 7 has the most of them, of 16 rows one of 8)
  static constexpr uint32_t kHalfBytes = (kTok == 16 ? 32 : kTok == 32 ? 56 : 84) * 128 * 4;
  static constexpr uint32_t kExchangeBytes = kHalves * kHalfBytes;
  static constexpr uint32_t kFactorBytes = kFactorSlots * kHalves * kTok * 4;
  static constexpr uint32_t kOther =
      kExchangeBytes + kFactorBytes + sizeof(ExpertTiles) + 4 * kTok * 4 + 512 + 1024;
  static constexpr int kStages = (int)((232448u - kOther) / kStageBytes) > 12
                                     ? 12
                                     : (int)((232448u - kOther) / kStageBytes);
  static_assert(kStages >= 3 && kTmemCols <= 512);
  static constexpr uint32_t kOffExchange = kStages * kStageBytes;
  static constexpr uint32_t kOffFactors = kOffExchange + kExchangeBytes;
  static constexpr uint32_t kOffTop = kOffFactors + kFactorBytes;
  static constexpr uint32_t kOffTiles = kOffTop + 4 * kTok * 4;
  static constexpr uint32_t kOffBars = (kOffTiles + sizeof(ExpertTiles) + 15) / 16 * 16;
  // full[kStages], empty[kStages], acc_full[kBufs], acc_empty[kBufs],
  // factor_full[slots], factor_empty[slots], exchange, drain
  static constexpr uint32_t kFull = 0, kEmpty = 8 * kStages;
  static constexpr uint32_t kAccFull = 16 * kStages, kAccEmpty = kAccFull + 8 * kBufs;
  static constexpr uint32_t kFactorFull = kAccEmpty + 8 * kBufs;
  static constexpr uint32_t kFactorEmpty = kFactorFull + 8 * kFactorSlots;
  static constexpr uint32_t kPeerFull = kFactorEmpty + 8 * kFactorSlots;
  static constexpr uint32_t kDrain = kPeerFull + 8;
  static constexpr int kBarriers = kDrain / 8 + 1;
  static constexpr uint32_t kTmemSlot = kDrain + 8, kAbort = kTmemSlot + 4;
  static_assert(kAbort + 4 <= 512);
  static constexpr size_t kBytes = kOffBars + 512 + 1024;  // room to align the base
  static_assert(kBytes <= 232448);
};

struct FewTile {
  int expert, row0, rows, block;
};

template <int kTok>
__device__ __forceinline__ FewTile few_tile(const MatmulParams& p, const ExpertTiles& s, int index) {
  FewTile t;
  t.expert = expert_of_tile(p, s, index);
  const int at = index - s.tile_start[t.expert];
  const int tiles = (s.rows(t.expert) + kTok - 1) / kTok;
  t.block = at / tiles;
  const int r = at - t.block * tiles;
  t.row0 = s.row_start[t.expert] + r * kTok;
  t.rows = min(kTok, s.rows(t.expert) - r * kTok);
  return t;
}

// What the summing warps know of their block.
struct FewBlock {
  uint8_t* sm;
  uint32_t base, bars, tmem, abort;
  int split, rank, first, stride, total, steps;
};

// The sums of every tile, one feature to a thread, and their way out.
template <int kTok, bool kGated>
__device__ __forceinline__ void sum_and_write(const MatmulParams& p, const ExpertTiles& tiles,
                                              const FewBlock& b) {
  using F = Few<kTok, kGated>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, quarter = warp & 3, feature = quarter * 32 + lane;
  const uint32_t from = b.tmem + ((uint32_t)(quarter * 32) << 16) + half * kTok;
  const int per = (kTok / 4 + b.split - 1) / b.split * 4;  // rows that a rank owns
  const uint32_t mine = F::kOffExchange + (uint32_t)half * F::kHalfBytes + feature * 16;
  float4* const exchange = reinterpret_cast<float4*>(b.sm + mine);
  float4* const exchange_up = reinterpret_cast<float4*>(b.sm + mine + F::kHalfBytes);
  const int own = b.rank * per / 4 * 128;
  uint32_t* const tops = reinterpret_cast<uint32_t*>(b.sm + F::kOffTop);
  uint32_t it = 0;
  bool ok = true, met = false;  // (a warp that gives up still takes part in the barriers)
#pragma unroll 1
  for (int index = b.first; index < b.total && (kGated || ok); index += b.stride) {
    const FewTile t = few_tile<kTok>(p, tiles, index);
    float acc[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) acc[i] = 0.0f;
#pragma unroll 1
    for (int step = 0; ok && step < b.steps;) {
      // (what precedes the last of a batch is complete when that is)
      const int batch = min(F::kBatch, b.steps - step);
      const uint32_t last = it + batch - 1;
      ok = uniform_wait2(b.bars + F::kFactorFull + 8 * (last % kFactorSlots), (last / kFactorSlots) & 1,
                         b.bars + F::kAccFull + 8 * (last % F::kBufs), (last / F::kBufs) & 1, b.abort);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < F::kBatch; ++j) {
        if (j >= batch) break;
        const int buf = (it + j) % F::kBufs, slot = (it + j) % kFactorSlots;
        const uint32_t factors =
            b.base + F::kOffFactors + (uint32_t)(slot * F::kHalves + half) * kTok * 4;
#pragma unroll
        for (int c = 0; c < kTok / 16; ++c) {
          if (16 * c < t.rows) {
            uint32_t v[16];
            uint4 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = lds_v4_at(factors + 64 * c + 16 * i);
            tmem_ld16(from + buf * F::kAccCols + 16 * c, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* a = acc + 16 * c + 4 * i;
              a[0] = fmaf(__uint_as_float(v[4 * i]), __uint_as_float(f[i].x), a[0]);
              a[1] = fmaf(__uint_as_float(v[4 * i + 1]), __uint_as_float(f[i].y), a[1]);
              a[2] = fmaf(__uint_as_float(v[4 * i + 2]), __uint_as_float(f[i].z), a[2]);
              a[3] = fmaf(__uint_as_float(v[4 * i + 3]), __uint_as_float(f[i].w), a[3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane < batch) {
        mbar_arrive(b.bars + F::kAccEmpty + 8 * ((it + lane) % F::kBufs));
        mbar_arrive(b.bars + F::kFactorEmpty + 8 * ((it + lane) % kFactorSlots));
      }
      __syncwarp();
      step += batch;
      it += batch;
    }
    // rows whose r lies outside a count as zeros
    uint64_t valid = 0;
#pragma unroll
    for (int i = 0; i < (kTok + 31) / 32; ++i) {
      bool in = lane + 32 * i < t.rows;
      if (in) a_row(p, t.row0 + lane + 32 * i, in);
      valid |= (uint64_t)__ballot_sync(0xFFFFFFFFu, in) << (32 * i);
    }
    const int r0 = b.rank * per;
    int rows = max(min(per, t.rows - r0), 0);
    if (b.split > 1) {  // (a cluster has one tile at most)
      cluster_wait_all();
      if (threadIdx.x == 0)
        mbar_expect_tx(b.bars + F::kPeerFull, (uint32_t)(b.split * ((rows + 3) / 4) * 2048 * F::kHalves));
      const uint32_t first = b.base + mine + own * 16;
      uint32_t to = 0, bar = 0;
      int owner = 0, left = 0;
#pragma unroll
      for (int i = 0; i < kTok; i += 4) {
        if (left == 0) {
          to = in_cluster(first, owner);
          bar = in_cluster(b.bars + F::kPeerFull, owner++);
          left = per;
        }
        if (ok && i < t.rows) st_async4(to, acc + i, bar);
        to += 128 * 16;
        left -= 4;
      }
      __syncwarp();
      cluster_arrive();
      met = true;
      ok = ok && cluster_wait(b.bars + F::kPeerFull, 0, b.abort);
    } else {
#pragma unroll
      for (int i = 0; i < kTok; i += 4)
        if (i < t.rows)
          exchange[i * 32] = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    }
    if (!ok) rows = 0;
    // four rows' sums over the ranks
    const auto sum = [&](int row) {
      float4 v = exchange[row * 32];
      for (int q = 1; q < b.split; ++q) {
        const float4 w = exchange[(q * per + row) * 32];
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      return v;
    };
    const int64_t first_row = t.row0 + r0;
    if (rows > 0) valid >>= r0;
    if constexpr (!kGated) {
      const int column = t.block * 128 + feature;
      if (column < p.n) {
        uint8_t* to = p.out + first_row * p.out_pitch + 2 * (int64_t)column;
#pragma unroll 2
        for (int row = 0; row < rows; row += 4) {
          const float4 v4 = sum(row);
          const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i, to += p.out_pitch) {
            const uint32_t w = narrow2_to(valid >> (row + i) & 1 ? v[i] : 0.0f, 0.0f, p.half != 0);
            if (row + i < rows)
              asm volatile("st.global.u16 [%0], %1;" ::"l"(to), "h"((uint16_t)w) : "memory");
          }
        }
      }
    } else {
      if (half == 1 && b.split > 1)
        for (int row = 0; row < rows; row += 4) exchange[own + row * 32] = sum(row);
      named_barrier(1, 256);
      if (half == 0) {
        for (int row = 0; row < rows; row += 4) {
          const float4 g = sum(row), u = exchange_up[own + row * 32];
          float z[4] = {gated(g.x, u.x), gated(g.y, u.y), gated(g.z, u.z), gated(g.w, u.w)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!(valid >> (row + i) & 1)) z[i] = 0.0f;
            const uint32_t top = __reduce_max_sync(
                0xFFFFFFFFu, z[i] == z[i] ? __float_as_uint(fabsf(z[i])) : 0u);
            if (lane == 0) tops[quarter * kTok + row + i] = top;
          }
          exchange[own + row * 32] = make_float4(z[0], z[1], z[2], z[3]);
        }
        named_barrier(2, 128);
        uint8_t* to = p.out + first_row * p.out_pitch + t.block * 128 + feature;
#pragma unroll 4
        for (int row = 0; row < rows; ++row, to += p.out_pitch) {
          const uint32_t top = max(max(tops[row], tops[kTok + row]),
                                   max(tops[2 * kTok + row], tops[3 * kTok + row]));
          const float most = __uint_as_float(top);
          const float z = reinterpret_cast<const float*>(exchange + own + row / 4 * 128)[row & 3];
          const uint32_t code = cvt_e4m3x2(z * code_factor(most), 0.0f);
          asm volatile("st.global.u8 [%0], %1;" ::"l"(to), "r"(code) : "memory");
          if (feature == 0)
            p.out_scales[(first_row + row) * p.out_scale_stride + t.block] = code_scale(most);
        }
      }
      named_barrier(1, 256);
    }
  }
  if (b.split > 1 && !met) {
    cluster_wait_all();
    cluster_arrive();
  }
}

template <int kTok, bool kGated>
__global__ void __launch_bounds__(Few<kTok, kGated>::kThreads, 1)
    fp8_matmul_few_kernel(const __grid_constant__ MatmulParams p, int split) {
  using F = Few<kTok, kGated>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  const uint32_t base = smem_addr(sm), bars = base + F::kOffBars;
  ExpertTiles& tiles = *reinterpret_cast<ExpertTiles*>(sm + F::kOffTiles);
  const uint32_t abort = bars + F::kAbort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;

  // this block's steps of every tile
  const int k0 = p.steps * rank / split, k1 = p.steps * (rank + 1) / split;
  const int first = blockIdx.x / split, stride = gridDim.x / split;
  const auto load_step = [&](const FewTile& t, int kb, int st) {
    const uint32_t full = bars + F::kFull + 8 * st, dst = base + st * F::kStageBytes;
    // (through an index no more rows come than there are, by fours)
    const uint32_t rows = p.rows ? (t.rows + 3) & ~3 : kTok;
    mbar_expect_tx(full, F::kHalves * F::kWeightBytes + rows * kGroupK);
    tma_load_3d(dst, &p.b_map, kb * kGroupK, t.block * 128, t.expert, full);
    if (kGated)
      tma_load_3d(dst + F::kWeightBytes, &p.b_map, kb * kGroupK, (t.block + p.up_blocks) * 128,
                  t.expert, full);
    if (!p.rows)
      tma_load_2d(dst + F::kHalves * F::kWeightBytes, &p.a_map, kb * kGroupK, t.row0, full);
  };
  int early = 0;  // steps of the first tile that are loaded already
  if (warp == F::kLoadWarp) {
    for (int i = lane; i < F::kBarriers; i += 32) {
      const int at = 8 * i;
      const int sums = (at >= F::kAccEmpty && at < F::kFactorFull) ||
                       (at >= F::kFactorEmpty && at < F::kPeerFull);
      mbar_init(bars + at, sums ? F::kSumWarps : 1);
    }
    if (lane == 0) *reinterpret_cast<volatile int*>(sm + F::kOffBars + F::kAbort) = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
    __syncwarp();
    // One matrix: the first tile is known before anything is counted, and its loads
    // travel while the block starts (with the meeting of the cluster's blocks
    // in two parts, 8 x 4096 x 6144 went from 10.9 to 9.6 us).
    if (!p.offsets) {
      const int tiles = (p.num_rows + kTok - 1) / kTok, block = first / tiles;
      const FewTile t{0, (first - block * tiles) * kTok, 0, block};
      early = min(k1 - k0, kEarly);
      if (elect_one())
        for (int i = 0; i < early; ++i) load_step(t, k0 + i, i);
      __syncwarp();
    }
  }
  if (warp == F::kMmaWarp) tmem_alloc(bars + F::kTmemSlot, F::kTmemCols);
  tc_fence_before();
  count_tiles<kTok, F::kThreads>(p, tiles);
  __syncthreads();
  // (the barriers are ready: waited for where the sums meet, or a role ends)
  if (split > 1) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + F::kOffBars + F::kTmemSlot);
  const int total = tiles.tile_start[p.experts];

  if (warp == F::kLoadWarp) {
    uint32_t it = early;
    bool ok = true;
    for (int index = first; ok && index < total; index += stride) {
      const FewTile t = few_tile<kTok>(p, tiles, index);
      int r[4] = {0, 0, 0, 0};
      if (4 * lane < t.rows && p.rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bool in;
          r[i] = a_row(p, t.row0 + min(4 * lane + i, t.rows - 1), in);
        }
      }
      for (int kb = k0 + (index == first ? early : 0); kb < k1; ++kb, ++it) {
        const int st = it % F::kStages;
        if (it >= F::kStages &&
            !uniform_wait(bars + F::kEmpty + 8 * st, (it / F::kStages - 1) & 1, abort)) {
          ok = false;
          break;
        }
        if (elect_one()) load_step(t, kb, st);
        __syncwarp();
        if (4 * lane < t.rows && p.rows)
          tma_gather4(base + st * F::kStageBytes + F::kHalves * F::kWeightBytes + lane * 4 * kGroupK,
                      &p.a_map, kb * kGroupK, r[0], r[1], r[2], r[3], bars + F::kFull + 8 * st);
      }
    }
    // copies that no MMA will wait for end before the block does
    if (gone(abort)) {
      for (uint32_t i = it > F::kStages ? it - F::kStages : 0; i < it; ++i)
        for (uint32_t n = 0;
             n < kWaitPolls && !mbar_test(bars + F::kFull + 8 * (i % F::kStages), (i / F::kStages) & 1);)
          ++n;
    }
  } else if (warp == F::kMmaWarp) {
    uint32_t it = 0;
    bool ok = true;
    for (int index = first; ok && index < total; index += stride) {
      const FewTile t = few_tile<kTok>(p, tiles, index);
      const uint32_t idesc = instr_desc_f8(128, (t.rows + 15) & ~15);
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int st = it % F::kStages, buf = it % F::kBufs;
        // (the first use of an accumulator passes: the phase before the first)
        ok = uniform_wait2(bars + F::kAccEmpty + 8 * buf, (it / F::kBufs + 1) & 1,
                           bars + F::kFull + 8 * st, (it / F::kStages) & 1, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = base + st * F::kStageBytes;
        const uint64_t rows = smem_desc(at + F::kHalves * F::kWeightBytes, 16, 1024, 2);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < F::kHalves; ++h) {
            const uint64_t weights = smem_desc(at + h * F::kWeightBytes, 16, 1024, 2);
            const uint32_t d = tmem + buf * F::kAccCols + h * kTok;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ss_f8(d, desc_at(weights, 32 * j), desc_at(rows, 32 * j), idesc, j > 0);
          }
          mma_commit(bars + F::kEmpty + 8 * st);
          mma_commit(bars + F::kAccFull + 8 * buf);
        }
        __syncwarp();
      }
    }
    // (bounded, abort or not: no MMA is left when the block ends)
    if (elect_one()) mma_commit(bars + F::kDrain);
    __syncwarp();
    bool drained = false;
    for (uint32_t i = 0; i < kWaitPolls && !drained; ++i) drained = mbar_test(bars + F::kDrain, 0);
    if (!drained) give_up(abort);
    __syncwarp();
  } else if (warp == F::kScaleWarp) {
    // sa[row][g] * sb[g] of a step, many steps' loads at a time: a trip to memory takes as
    // long as four steps or more
    constexpr int kRowsPer = (kTok + 31) / 32;
    constexpr int kAhead = kRowsPer == 1 ? 16 : kGated ? 4 : 8;
    uint32_t it = 0;
    bool ok = true;
    for (int index = first; ok && index < total; index += stride) {
      const FewTile t = few_tile<kTok>(p, tiles, index);
      const float* sa[kRowsPer];
      bool in[kRowsPer];
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) {
        const int row = lane + 32 * i;
        in[i] = row < t.rows;
        sa[i] = p.a_scales;
        if (in[i]) sa[i] += a_row(p, t.row0 + row, in[i]) * p.a_scale_stride;
      }
      const float* sb = p.b_scales + t.expert * p.b_scale_expert_stride + t.block * p.b_scale_stride;
      const float* sb_up = sb + p.up_blocks * p.b_scale_stride;
      float x[kRowsPer][kAhead], w[kAhead], u[kAhead];
      const auto load = [&](int kb) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const bool have = kb + j < k1;
          w[j] = have ? ld_f32(sb + kb + j) : 0.0f;
          u[j] = kGated && have ? ld_f32(sb_up + kb + j) : 0.0f;
#pragma unroll
          for (int i = 0; i < kRowsPer; ++i)
            x[i][j] = have && in[i] ? ld_f32(sa[i] + (int64_t)(kb + j) * p.a_group_step) : 0.0f;
        }
      };
      load(k0);
      for (int kb = k0; ok && kb < k1; kb += kAhead) {
        float f[F::kHalves][kRowsPer][kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int i = 0; i < kRowsPer; ++i) {
            f[0][i][j] = x[i][j] * w[j];
            if (kGated) f[F::kHalves - 1][i][j] = x[i][j] * u[j];
          }
        if (kb + kAhead < k1) load(kb + kAhead);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (kb + j >= k1 || !ok) break;
          const int slot = it % kFactorSlots;
          if (it >= kFactorSlots &&
              !uniform_wait(bars + F::kFactorEmpty + 8 * slot, (it / kFactorSlots - 1) & 1, abort)) {
            ok = false;
            break;
          }
          float* to = reinterpret_cast<float*>(sm + F::kOffFactors) + slot * F::kHalves * kTok;
#pragma unroll
          for (int i = 0; i < kRowsPer; ++i)
            if (lane + 32 * i < kTok) {
#pragma unroll
              for (int h = 0; h < F::kHalves; ++h) to[h * kTok + lane + 32 * i] = f[h][i][j];
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + F::kFactorFull + 8 * slot);
          ++it;
        }
      }
    }
  } else {
    const FewBlock b{sm, base, bars, tmem, abort, split, rank, first, stride, total, k1 - k0};
    sum_and_write<kTok, kGated>(p, tiles, b);
  }
  if (split > 1 && warp >= F::kSumWarps) {
    __syncwarp();
    cluster_wait_all();
    cluster_arrive();
  }
  __syncthreads();
  const bool aborted = *reinterpret_cast<volatile int*>(sm + F::kOffBars + F::kAbort) != 0;
  if (tid == 0 && aborted && p.status) atomicExch(p.status, 1);
  // No block leaves while another one may still write to it: it has waited for the
  // others' sums, or, given up, waits a while for them here.
  if (split > 1) {
    if (aborted)
      for (uint32_t i = 0; i < kWaitPolls && !mbar_test(bars + F::kPeerFull, 0);) ++i;
    __syncwarp();
    cluster_wait_all();
  }
  if (warp == F::kMmaWarp) tmem_dealloc(tmem, F::kTmemCols);
}

// Clusters of the kernel that run at once on the current device, 0: none (and,
// once for each device, the kernel's permission to use that much shared memory).
template <int kTok, bool kGated>
int resident_clusters(int split) {
  using F = Few<kTok, kGated>;
  const auto kernel = fp8_matmul_few_kernel<kTok, kGated>;
  static int cache[64][kMostSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int& n = cache[dev][split];
  if (n) return n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::kBytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (split == 1) return n = sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split);
  cfg.blockDim = dim3(F::kThreads);
  cfg.dynamicSmemBytes = F::kBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int found = 0;
  if (cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n = found;
}

template <int kTok, bool kGated>
int launch(const MatmulParams& p, cudaStream_t stream) {
  using F = Few<kTok, kGated>;
  // at most this many tiles: every expert's last tile of rows may be a short one
  const int64_t row_tiles =
      p.offsets ? (int64_t)p.num_rows / kTok + (p.num_rows < p.experts ? p.num_rows : p.experts)
                : p.row_tiles_dense;
  const int64_t most = row_tiles * p.column_tiles;
  int split = 1;
  int64_t room = resident_clusters<kTok, kGated>(1);
  if (room == 0) return KVQ_ECUDA;
  for (int s = 2; s <= kMostSplit && s <= p.steps && most * s <= sm_count(); ++s) {
    const int64_t r = resident_clusters<kTok, kGated>(s);
    if (r < most) continue;
    split = s;
    room = r;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((most < room ? most : room) * split));
  cfg.blockDim = dim3(F::kThreads);
  cfg.dynamicSmemBytes = F::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fp8_matmul_few_kernel<kTok, kGated>, p, split) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  return launch_status();
}

}  // namespace

// row_tile 16, 32 or 64.
int launch_matmul_few(const MatmulParams& p, bool is_gated, int row_tile, cudaStream_t stream) {
  if (is_gated)
    return row_tile == 16   ? launch<16, true>(p, stream)
           : row_tile == 32 ? launch<32, true>(p, stream)
                            : launch<64, true>(p, stream);
  return row_tile == 16   ? launch<16, false>(p, stream)
         : row_tile == 32 ? launch<32, false>(p, stream)
                          : launch<64, false>(p, stream);
}

}  // namespace kvq
