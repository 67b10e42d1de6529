// fp8_matmul_tiles.cu — the kernel of the block-scaled 8-bit products for many
// rows to a matrix.
//
//   out[i][j] = sum_g sa[i][g] sb[j/128][g] sum_{l in g} a[i][l] b[j][l]
//
// A pair of blocks (cta_group::2) takes a tile of 256 of a's rows, the M side of
// tcgen05.mma, and 256 of b's rows, columns of the result, its N side. A step is a
// group of 128 values: each block loads 128 rows of both, 32 KB, for 512 cycles of the
// tensor cores at their rate; four MMAs form the group's product in one of two
// accumulators (256 columns each, all of tensor memory), and eight warps add it,
// scaled, to sums in registers while the next one is formed:
//   acc[j] += partial[j] * (sa sb).
// A thread has one row and 128 columns, which are one block of b: one factor for a
// step, which two warps bring to shared memory ahead (loaded by the sums themselves they
// cost a tenth of the time). (The product the other way round,
// rows as the N side, needs no more than 32 rows to a step of the tile, but a factor for
// every fourth column: its sums took 1.5 times as long, and set the pace.)
//
// Gated: a half is 64 columns of the gate's block and the 64 of the up block that belong
// to them; the two threads of a row exchange their largest value. (A half for each took an
// exchange of 64 sums a thread, 5000 cycles a tile with the rest of its end.)
//
// Rows through an index come by 16-byte asynchronous copies of four more warps: a TMA
// gather moves four rows of 128 bytes at 95 cycles an instruction. (By the two
// warps of the factors 880 cycles a step: 32768 rows of 64 gated experts, 4096 -> 1024,
// took 323 us and take 281, in place 261.)
//
// Roles: warps 0-7 sums (32 rows by warp % 4, half of the columns by warp / 4), 8 TMA, 9
// MMA (of the first block), 10 and 11 factors, 12-15 rows through an index. Tiles are taken
// in turn by resident pairs; loads and products run ahead over a tile's end.
//
// Bound by the sums, 700 cycles a step of 256 columns (the tensor cores are busy for 512): 8192 x
// 7168 x 4096 takes 161 us, 2980 TFLOP/s; a tile's end, 1 to 2 us, weighs more the shorter
// k is (32768 rows of 64 experts, 1024 -> 4096: 154 us).
#include <cstddef>

#include "fp8_matmul.cuh"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kTileRows = 256;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kFactorWarp = 10, kCopyWarp = 12;
// Threads, and registers of a thread: 168 or 128 at launch, handed to the sums. The
// compiler takes what is handed out for its limit, and at other splits it spills in the
// sums' loop: 8192 x 7168 x 4096 took 161 us with 216, 209 to 211 with 200, 208 and 224;
// rows through an index, gated, 276 us with 216, 345 with 208, 350 with 200.
template <bool kIndex>
struct Warps {
  static constexpr int kThreads = kIndex ? 512 : 384;
  static constexpr int kSums = 216;
  static constexpr int kOthers = kIndex ? 40 : 72;
  static_assert(256 * kSums + (kThreads - 256) * kOthers <= kThreads * (kIndex ? 128 : 168));
};

// Stages of a step's loads; where tiles leave by bulk stores, the last two's room holds
// the tile instead (8192 x 7168 x 4096 takes 161 us; 167 with six and stores by the
// threads, 170 with four).
constexpr int kMostStages = 6;
template <bool kGated, bool kAligned>
constexpr int kStagesOf = !kGated && kAligned ? 4 : kMostStages;
constexpr uint32_t kHalf = 128 * kGroupK;  // a block's rows of a, or of b
constexpr uint32_t kStageBytes = 2 * kHalf;
// gated, and rows of any alignment: 2 KB of each warp of the sums, on their way out
constexpr uint32_t kExchangeBytes = 16384;
constexpr uint32_t kOffTile = 4 * kStageBytes;  // of each warp of the sums 2 x 32 rows of 128 bytes
constexpr uint32_t kOffExchange = kMostStages * kStageBytes;
// factors: [slot][step of a group][half of the columns][row]
constexpr int kGroup = 2, kSlots = 4;
constexpr uint32_t kStepFactors = 2 * 128 * 4;
constexpr uint32_t kOffFactors = kOffExchange + kExchangeBytes;
// what the sums need to know of a tile: where it lies, and which rows of a exist
struct TileNote {
  int row0, rows, column, unused;
  uint32_t valid[4];
};
constexpr int kNotes = 8;  // (factors are at most kSlots tiles ahead of the sums)
constexpr uint32_t kOffNotes = kOffFactors + kSlots * kGroup * kStepFactors;
constexpr uint32_t kOffTiles = kOffNotes + kNotes * sizeof(TileNote);
constexpr uint32_t kOffBars = (kOffTiles + sizeof(ExpertTiles) + 15) / 16 * 16;
constexpr uint32_t kFull = 0, kEmpty = 8 * kMostStages;
constexpr uint32_t kAccFull = 16 * kMostStages, kAccEmpty = kAccFull + 16;
constexpr uint32_t kFactorFull = kAccEmpty + 16, kFactorEmpty = kFactorFull + 8 * kSlots;
constexpr uint32_t kCopied = kFactorEmpty + 8 * kSlots, kDrain = kCopied + 8 * kMostStages;
constexpr uint32_t kTmemSlot = kDrain + 8, kAbort = kTmemSlot + 4, kTotal = kAbort + 4;
static_assert(kTotal + 4 <= 512);
constexpr size_t kBytes = kOffBars + 512 + 1024;  // room to align the base
static_assert(kBytes <= 232448);

// ------------------------------------------------------ pairs of blocks ---

__device__ __forceinline__ void pair_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}
// 256 x N x 32 of E4M3 by both blocks of a pair; one thread of the first.
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both blocks once every MMA issued so far has completed.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// An arrival on a barrier of the pair's first block, with no data of shared memory.
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// An arrival there behind rows that threads of this block have written to its shared memory,
// and what the first block's issuer does before its products, asynchronous, read them. (A fence
// of nothing but shared memory: as a release of the whole cluster, 1700 cycles each, 32768
// rows of 64 gated experts, 4096 -> 1024, took 520 us, by this one 280.)
__device__ __forceinline__ void arrive_rows(uint32_t bar) {
  asm volatile("fence.proxy.async::generic.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void acquire_rows() {
  asm volatile("fence.proxy.async::generic.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
// As mbar_test, of arrive_rows' arrivals, with acquire_rows to follow.
__device__ __forceinline__ bool mbar_test_rows(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Loads into this block that complete on a barrier of the pair's first.
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                             int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// ------------------------------------------------------------------ tiles ---

// Tiles go down bands of kBand tiles' rows, column by column: what the pairs read at once is
// less than whole columns of many rows (16384 x 4096 x 4096 by whole columns 213 us, by
// bands of 4 to 16 tiles 209 to 200).
constexpr int kBand = 16;

struct PairTile {
  int expert, row0, rows, column;
};

__device__ __forceinline__ PairTile pair_tile(const MatmulParams& p, const ExpertTiles& s,
                                              int index) {
  PairTile t;
  t.expert = expert_of_tile(p, s, index);
  const int at = index - s.tile_start[t.expert];
  const int tiles = (s.rows(t.expert) + kTileRows - 1) / kTileRows;
  const int band = at / (kBand * p.column_tiles), within = at - band * kBand * p.column_tiles;
  const int height = min(kBand, tiles - kBand * band);
  t.column = within / height;
  const int r = kBand * band + within - t.column * height;
  t.row0 = s.row_start[t.expert] + r * kTileRows;
  t.rows = min(kTileRows, s.rows(t.expert) - r * kTileRows);
  return t;
}

struct PairBlock {
  uint8_t* sm;
  uint32_t base, bars, tmem, abort;
  int rank, first, stride, total;
};

// Tells the pair's first block that this one's copied rows of a step are there.
template <int kStages>
__device__ __forceinline__ bool announce_rows(const PairBlock& b, uint32_t it) {
  const int st = it % kStages;
  if (!uniform_wait(b.bars + kCopied + 8 * st, (it / kStages) & 1, b.abort)) return false;
  if (elect_one()) arrive_rows(in_cluster(b.bars + kFull + 8 * st, 0));
  __syncwarp();
  return true;
}

// Rows through an index are announced kLag steps behind: later than they come, and early
// enough for the products. (Gated, with six stages, 279 us one step behind, 283 two, 286 three;
// 32768 rows of 64 experts, 4096 -> 2048, with four stages 285, 280 and 417.)
template <bool kGated>
constexpr uint32_t kLagOf = kGated ? 1 : 2;

template <int kStages, bool kGated, bool kIndex>
__device__ __forceinline__ void load_tiles(const MatmulParams& p, const ExpertTiles& tiles,
                                           const PairBlock& b) {
  constexpr uint32_t kLag = kLagOf<kGated>;
  uint32_t it = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride) {
    const PairTile t = pair_tile(p, tiles, index);
    const int column = kGated ? t.column * 128 + b.rank * 64 : t.column * 256 + b.rank * 128;
    for (int kb = 0; kb < p.steps; ++kb, ++it) {
      const int st = it % kStages;
      if (it >= kStages &&
          !uniform_wait(b.bars + kEmpty + 8 * st, (it / kStages - 1) & 1, b.abort)) {
        ok = false;
        break;
      }
      const uint32_t dst = b.base + st * kStageBytes;
      const uint32_t full = in_cluster(b.bars + kFull + 8 * st, 0);
      if (elect_one()) {
        if (b.rank == 0) mbar_expect_tx(b.bars + kFull + 8 * st, kIndex ? 2 * kHalf : 4 * kHalf);
        if (!kIndex)
          pair_load_2d(dst, &p.a_map, kb * kGroupK, t.row0 + b.rank * 128, full);
        pair_load_3d(dst + kHalf, &p.b_map, kb * kGroupK, column, t.expert, full);
        if (kGated)
          pair_load_3d(dst + kHalf + kHalf / 2, &p.b_map, kb * kGroupK, column + p.up_blocks * 128,
                       t.expert, full);
      }
      __syncwarp();
      if (kIndex && it >= kLag && !announce_rows<kStages>(b, it - kLag)) {
        ok = false;
        ++it;
        break;
      }
    }
  }
  if (kIndex)
    for (uint32_t i = it > kLag ? it - kLag : 0; ok && i < it; ++i) ok = announce_rows<kStages>(b, i);
  // the first block's arrivals here end before this block does
  for (uint32_t i = it > kStages ? it - kStages : 0; ok && i < it; ++i)
    ok = uniform_wait(b.bars + kEmpty + 8 * (i % kStages), (i / kStages) & 1, b.abort);
  // copies that no MMA will wait for end before the pair does
  if (b.rank == 0 && gone(b.abort)) {
    for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
      for (uint32_t n = 0;
           n < kWaitPolls && !mbar_test(b.bars + kFull + 8 * (i % kStages), (i / kStages) & 1);)
        ++n;
  }
}

__device__ __forceinline__ void cp_async_16_at(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 16 bytes, or zeros.
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const uint8_t* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(have ? 16 : 0)
               : "memory");
}

// Two warps, 64 of this block's 128 rows each: sa[row] * sb of both halves of the
// columns for every step, a group of steps at a time, the next group's loads under way.
template <bool kGated>
__device__ __forceinline__ void serve_factors(const MatmulParams& p, const ExpertTiles& tiles,
                                              const PairBlock& b) {
  const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) - kFactorWarp;
  const bool vector = p.a_group_step != 0 && p.a_scale_stride % 2 == 0 &&
                      (reinterpret_cast<uintptr_t>(p.a_scales) & 7) == 0;
  float* const to = reinterpret_cast<float*>(b.sm + kOffFactors) + part * 64 + lane;
  uint32_t group = 0, count = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride, ++count) {
    const PairTile t = pair_tile(p, tiles, index);
    const int row0 = b.rank * 128 + part * 64;  // of the tile
    TileNote* const note = reinterpret_cast<TileNote*>(b.sm + kOffNotes) + count % kNotes;
    const float* sa[2];                         // null: no such row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bool in = row0 + lane + 32 * i < t.rows;
      const int64_t at = in ? a_row(p, t.row0 + row0 + lane + 32 * i, in) : 0;
      sa[i] = in ? p.a_scales + at * p.a_scale_stride : nullptr;
      const uint32_t valid = __ballot_sync(0xFFFFFFFFu, in);
      if (lane == 0) note->valid[2 * part + i] = valid;
    }
    if (part == 0 && lane == 0) {
      note->row0 = t.row0;
      note->rows = t.rows;
      note->column = t.column;
    }
    __syncwarp();  // (read behind the first factors' arrival)
    const float* sb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sb[h] = p.b_scales + t.expert * p.b_scale_expert_stride +
              (kGated ? t.column + h * p.up_blocks : min(2 * t.column + h, p.blocks - 1)) *
                  p.b_scale_stride;
    float x[2][kGroup], w[2][kGroup];
    const auto load = [&](int kb) {
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h][j] = kb + j < p.steps ? ld_f32(sb[h] + kb + j) : 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (vector && kb + kGroup <= p.steps) {
          const float2 v = sa[i] ? __ldg(reinterpret_cast<const float2*>(sa[i] + kb)) : make_float2(0.0f, 0.0f);
          x[i][0] = v.x;
          x[i][1] = v.y;
        } else {
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            x[i][j] = sa[i] && kb + j < p.steps ? ld_f32(sa[i] + (kb + j) * p.a_group_step) : 0.0f;
        }
      }
    };
    load(0);
    for (int kb = 0; kb < p.steps; kb += kGroup) {
      const int slot = group % kSlots;
      if (group >= kSlots && !uniform_wait(b.bars + kFactorEmpty + 8 * slot,
                                           (group / kSlots - 1) & 1, b.abort)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            to[(slot * kGroup + j) * 256 + h * 128 + 32 * i] = x[i][j] * w[h][j];
      __syncwarp();
      if (elect_one()) mbar_arrive(b.bars + kFactorFull + 8 * slot);
      ++group;
      if (kb + kGroup < p.steps) load(kb + kGroup);
    }
  }
}

// Rows through an index: four warps, 32 of this block's 128 rows each, eight lanes to a row.
template <int kStages>
__device__ __forceinline__ void copy_rows(const MatmulParams& p, const ExpertTiles& tiles,
                                          const PairBlock& b) {
  const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) - kCopyWarp;
  const int sub = lane >> 3, piece = lane & 7;
  uint32_t it = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride) {
    const PairTile t = pair_tile(p, tiles, index);
    // (a row that does not exist: the last one, left out when the result is written)
    const uint8_t* from[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool in;
      const int64_t at =
          a_row(p, t.row0 + min(b.rank * 128 + part * 32 + 4 * i + sub, t.rows - 1), in);
      from[i] = p.a + at * p.a_stride + 16 * piece;
    }
    for (int kb = 0; kb < p.steps; ++kb, ++it) {
      const int st = it % kStages;
      if (it >= kStages &&
          !uniform_wait(b.bars + kEmpty + 8 * st, (it / kStages - 1) & 1, b.abort)) {
        ok = false;
        break;
      }
      // (rows of 128 bytes, pieces swizzled by row % 8)
      const uint32_t dst = b.base + st * kStageBytes + part * 32 * kGroupK + sub * kGroupK;
      const uint32_t even = dst + ((piece ^ sub) << 4), odd = dst + 4 * kGroupK + ((piece ^ (4 + sub)) << 4);
      if ((kb + 1) * kGroupK <= p.k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cp_async_16_at((i & 1 ? odd : even) + (i / 2) * 8 * kGroupK, from[i]);
          from[i] += kGroupK;
        }
      } else {
        const bool in_k = kb * kGroupK + 16 * piece < p.k;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          copy_or_zero((i & 1 ? odd : even) + (i / 2) * 8 * kGroupK, in_k ? from[i] : p.a, in_k);
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(b.bars + kCopied + 8 * st)
                   : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// uniform_wait2 of the issuer: for an accumulator, and for a step's operands, rows that the pair's
// second block has copied itself among them.
template <bool kIndex>
__device__ __forceinline__ bool wait_operands(uint32_t acc, uint32_t acc_parity, uint32_t full,
                                              uint32_t parity, uint32_t abort) {
  if constexpr (!kIndex) return uniform_wait2(acc, acc_parity, full, parity, abort);
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    const bool da = mbar_test(acc, acc_parity), db = mbar_test_rows(full, parity);
    if (__all_sync(0xFFFFFFFFu, da && db)) {
      acquire_rows();
      return true;
    }
    if ((i & 31u) == 31u && gone(abort)) return false;
  }
  give_up(abort);
  return false;
}

template <int kStages, bool kIndex>
__device__ __forceinline__ void issue_tiles(const MatmulParams& p, const PairBlock& b) {
  const uint32_t idesc = instr_desc_f8(256, 256);
  uint32_t it = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride) {
    for (int kb = 0; kb < p.steps; ++kb, ++it) {
      const int st = it % kStages, buf = it & 1;
      // (the first use of an accumulator passes: the phase before the first)
      ok = wait_operands<kIndex>(b.bars + kAccEmpty + 8 * buf, (it / 2 + 1) & 1,
                                 b.bars + kFull + 8 * st, (it / kStages) & 1, b.abort);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = b.base + st * kStageBytes;
      const uint64_t rows = smem_desc(at, 16, 1024, 2);
      const uint64_t columns = smem_desc(at + kHalf, 16, 1024, 2);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          pair_mma(b.tmem + buf * 256, desc_at(rows, 32 * j), desc_at(columns, 32 * j), idesc, j > 0);
        pair_commit(b.bars + kEmpty + 8 * st);
        pair_commit(b.bars + kAccFull + 8 * buf);
      }
      __syncwarp();
    }
  }
  // (bounded, abort or not: no MMA is left when the pair ends)
  if (elect_one())
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            b.bars + kDrain)
        : "memory");
  __syncwarp();
  for (uint32_t i = 0; i < kWaitPolls; ++i)
    if (mbar_test(b.bars + kDrain, 0)) return;
  give_up(b.abort);
}

// ------------------------------------------------------------------- sums ---

// A tile's steps: acc += partial * sa sb for the thread's row and 128 columns (kAny: the
// warp has rows). Nothing else lives in this loop: its registers are all taken, and one
// spilled costs a trip to L2.
template <bool kGated, bool kIndex, bool kAny>
__device__ __forceinline__ bool sum_steps(const MatmulParams& p, uint32_t base, uint32_t tmem,
                                          uint32_t& it, uint32_t& group, float (&acc)[4][32]) {
  const int quarter = threadIdx.x >> 5 & 3, half = threadIdx.x >> 7;
  const uint32_t bars = base + kOffBars;
  const uint32_t from0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
  const uint32_t factors = base + kOffFactors + (kGated ? threadIdx.x & 127 : threadIdx.x) * 4;
  const uint32_t to_leader = in_cluster(bars + kAccEmpty, 0);
  // (Through an index without a gate the next step's barriers are looked at while this
  // one's last columns are added, which takes 57 cycles each: 301 -> 282 us for 32768 rows of 64
  // experts, 4096 -> 2048. The other kernels gain nothing or lose: 166 -> 177 us.)
  bool ready = false;
#pragma unroll 1
  for (int kb = 0; kb < p.steps; ++kb, ++it) {
    const uint32_t slot = group % kSlots;
    if (!ready && !uniform_wait2(bars + kFactorFull + 8 * slot, (group / kSlots) & 1,
                                 bars + kAccFull + 8 * (it & 1), (it / 2) & 1, bars + kAbort))
      return false;
    tc_fence_after();
    const uint32_t from = from0 + (it & 1) * 256;
    float f[2] = {0.0f, 0.0f};
    if (kAny) {
      const uint32_t at = factors + (slot * kGroup + kb % kGroup) * kStepFactors;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[0]) : "r"(at) : "memory");
      f[1] = f[0];
      if (kGated) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[1]) : "r"(at + 512) : "memory");
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t v[32];
      if (kAny) tmem_ld32(from + 32 * c, v);
      if (c == 3) {
        tc_fence_before();
        __syncwarp();
        if (elect_one()) arrive_pair(to_leader + 8 * (it & 1));
        if constexpr (kIndex && !kGated) {
          const uint32_t then = (kb + 1) % kGroup == 0 ? group + 1 : group;
          const bool factors_there =
              mbar_test(bars + kFactorFull + 8 * (then % kSlots), (then / kSlots) & 1);
          ready = mbar_test(bars + kAccFull + 8 * (~it & 1), ((it + 1) / 2) & 1) && factors_there;
        }
      }
      if (kAny) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 r = fma2_rn({__uint_as_float(v[i]), __uint_as_float(v[i + 1])}, {f[c / 2], f[c / 2]},
                                   {acc[c][i], acc[c][i + 1]});
          acc[c][i] = r.x;
          acc[c][i + 1] = r.y;
        }
      }
    }
    if constexpr (kIndex && !kGated) ready = __all_sync(0xFFFFFFFFu, ready);
    if (kb % kGroup == kGroup - 1 || kb == p.steps - 1) {
      __syncwarp();
      if (elect_one()) mbar_arrive(bars + kFactorEmpty + 8 * slot);
      ++group;
    }
  }
  return true;
}

// A box of the result from shared memory.
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, uint32_t from) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(from)
               : "memory");
}

// `rows` of a warp's 32 rows, whose rows are aligned, to the warp's place in shared memory
// (`mine`: two halves of 64 columns, 16 bytes swizzled by row) and from there by two bulk
// stores, which go on beside the next tile: all pairs write at the same time, and by the
// threads' own stores that took 3000 cycles a tile. Fewer than 32 rows go by lanes: what
// lies behind them is another expert's.
__device__ __forceinline__ void send_rows(const MatmulParams& p, int64_t row, int rows, int column,
                                          uint32_t mine, const float (&acc)[4][32]) {
  const int lane = threadIdx.x & 31;
  if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float* a = &acc[k / 4][8 * (k % 4)];
    sts_v4(mine + k / 8 * 4096 + lane * 128 + ((k % 8 ^ (lane & 7)) << 4),
           make_uint4(narrow2_to(a[0], a[1], p.half != 0), narrow2_to(a[2], a[3], p.half != 0),
                      narrow2_to(a[4], a[5], p.half != 0), narrow2_to(a[6], a[7], p.half != 0)));
  }
  fence_proxy_async();
  __syncwarp();
  if (rows < 32) {
    uint8_t* to = p.out + row * p.out_pitch + 2 * (int64_t)column + 8 * lane;
#pragma unroll 1
    for (int r = 0; r < rows; ++r, to += p.out_pitch) {
      uint32_t x, y;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                   : "=r"(x), "=r"(y)
                   : "r"(mine + (lane >> 4) * 4096 + r * 128 + (((lane >> 1 & 7) ^ (r & 7)) << 4) +
                         (lane & 1) * 8)
                   : "memory");
      asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(to), "r"(x), "r"(y) : "memory");
    }
  } else if (elect_one()) {
#pragma unroll
    for (int h = 0; h < 2; ++h) store_box(&p.out_map, column + 64 * h, (int)row, mine + 4096 * h);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  __syncwarp();
}

// The same for 32 rows of any alignment and columns behind which the result ends: 32
// columns at a time through shared memory (2 KB of the warp's at `mine`, 16 bytes
// swizzled by row), a row by all lanes. (By its own thread 333 x 7001 took 58 us.)
__device__ __forceinline__ void write_rows_by_lanes(const MatmulParams& p, int64_t row, int rows,
                                                    int column, uint32_t mine,
                                                    const float (&acc)[4][32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* a = &acc[c][8 * k];
      sts_v4(mine + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4),
             make_uint4(narrow2_to(a[0], a[1], p.half != 0), narrow2_to(a[2], a[3], p.half != 0),
                        narrow2_to(a[4], a[5], p.half != 0), narrow2_to(a[6], a[7], p.half != 0)));
    }
    __syncwarp();
    const int at = column + 32 * c + lane;
    if (at < p.n) {
      uint8_t* to = p.out + row * p.out_pitch + 2 * (int64_t)at;
#pragma unroll 4
      for (int r = 0; r < rows; ++r, to += p.out_pitch) {
        uint16_t w;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(w)
                     : "r"(mine + r * 64 + (((lane >> 3) ^ (r >> 1 & 3)) << 4) + (lane & 7) * 2)
                     : "memory");
        asm volatile("st.global.u16 [%0], %1;" ::"l"(to), "h"(w) : "memory");
      }
    }
    __syncwarp();
  }
}

// The gated values of the thread's 64 columns and their codes; called by both warps of 32
// rows, of which `rows` exist. `mine` and `theirs`: 2 KB of each warp, first for the two
// threads of a row to leave their largest, then for the codes, which leave as rows do in
// send_rows.
__device__ __forceinline__ void write_gated(const MatmulParams& p, int64_t row, int rows, int block,
                                            uint32_t mine, uint32_t theirs, int half, int barrier,
                                            float (&acc)[4][32]) {
  const int lane = threadIdx.x & 31;
  if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
  float most = 0.0f;  // (fmaxf leaves NaN out)
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    float& z = acc[i / 32][i % 32];
    z = gated(z, acc[2 + i / 32][i % 32]);
    most = fmaxf(most, fabsf(z));
  }
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + lane * 4), "f"(most) : "memory");
  named_barrier(barrier, 64);
  float other;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(theirs + lane * 4) : "memory");
  named_barrier(barrier, 64);
  most = fmaxf(most, other);
  const float to_code = code_factor(most);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* z = &acc[i / 2][16 * (i & 1)];
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = cvt_e4m3x2(z[4 * k] * to_code, z[4 * k + 1] * to_code) |
             cvt_e4m3x2(z[4 * k + 2] * to_code, z[4 * k + 3] * to_code) << 16;
    sts_v4(mine + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  }
  if (half == 0 && lane < rows) p.out_scales[(row + lane) * p.out_scale_stride + block] = code_scale(most);
  fence_proxy_async();
  __syncwarp();
  const int column = block * 128 + half * 64;
  if (rows == 32) {
    if (elect_one()) {
      store_box(&p.out_map, column, (int)row, mine);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  } else if (lane < 16) {
    uint8_t* to = p.out + row * p.out_pitch + column + 4 * lane;
#pragma unroll 1
    for (int r = 0; r < rows; ++r, to += p.out_pitch) {
      uint32_t w;
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(w)
                   : "r"(mine + r * 64 + (((lane >> 2) ^ (r >> 1 & 3)) << 4) + (lane & 3) * 4)
                   : "memory");
      asm volatile("st.global.b32 [%0], %1;" ::"l"(to), "r"(w) : "memory");
    }
  }
  __syncwarp();
}

__device__ __forceinline__ int lds_int(uint32_t a) {
  int v;
  asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The sums of every tile and their way out. (What the loop over the steps does not need
// is read again behind it.)
template <bool kGated, bool kIndex, bool kAligned>
__device__ __forceinline__ void sum_tiles(const MatmulParams& p, uint32_t base, uint32_t tmem) {
  uint32_t it = 0, group = 0, count = 0;
  bool ok = true;  // (a warp that gives up still takes part in the warps' barriers)
#pragma unroll 1
  for (;; ++count) {
    const int index = blockIdx.x / 2 + count * (gridDim.x / 2);
    if (__all_sync(0xFFFFFFFFu, index >= lds_int(base + kOffBars + kTotal))) break;
    const uint32_t note = base + kOffNotes + count % kNotes * sizeof(TileNote);
    float acc[4][32];
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i / 32][i % 32] = 0.0f;
    if (ok)
      ok = uniform_wait(base + kOffBars + kFactorFull + 8 * (group % kSlots), (group / kSlots) & 1,
                        base + kOffBars + kAbort);
    if (ok) {
      const int rows = lds_int(note + offsetof(TileNote, rows)) - (int)cluster_rank() * 128;
      if (__any_sync(0xFFFFFFFFu, (int)(threadIdx.x & 127) < rows))
        ok = sum_steps<kGated, kIndex, true>(p, base, tmem, it, group, acc);
      else
        ok = sum_steps<kGated, kIndex, false>(p, base, tmem, it, group, acc);
    }
    const uint32_t again = base + kOffNotes + count % kNotes * sizeof(TileNote);
    const int half = threadIdx.x >> 7, row = (int)cluster_rank() * 128 + (threadIdx.x & 127);
    const bool have = ok && row < lds_int(again + offsetof(TileNote, rows));
    const int64_t to = (int64_t)lds_int(again + offsetof(TileNote, row0)) + row;
    const int column = lds_int(again + offsetof(TileNote, column));
    // a row that a does not have counts as zeros, whatever stood in for it
    const int valid = lds_int(again + offsetof(TileNote, valid) + (threadIdx.x >> 5 & 3) * 4);
    if (!(valid >> (threadIdx.x & 31) & 1)) {
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i / 32][i % 32] = 0.0f;
    }
    // (a vote: a branch that the compiler takes for divergent costs the loop over the
    // steps its uniform registers, and spills)
    if constexpr (kGated) {
      const int rows = __popc(__ballot_sync(0xFFFFFFFFu, have));
      const uint32_t at = base + kOffExchange, warp = threadIdx.x >> 5;
      write_gated(p, to - (row & 31), rows, column, at + warp * 2048, at + (warp ^ 4) * 2048, half,
                  1 + (warp & 3), acc);
    } else {
      const int at = column * 256 + half * 128;
      const int rows = __popc(__ballot_sync(0xFFFFFFFFu, have && at < p.n));
      if (rows > 0) {
        if (kAligned)
          send_rows(p, to - (row & 31), rows, at, base + kOffTile + (threadIdx.x >> 5) * 8192, acc);
        else
          write_rows_by_lanes(p, to - (row & 31), rows, at,
                              base + kOffExchange + (threadIdx.x >> 5) * 2048, acc);
      }
      if (!ok) break;
    }
  }
  if (kAligned && elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncwarp();
}

// kIndex: rows through an index. kAligned (not gated): out's rows are aligned and n is
// whole blocks of columns. (Kernels of their own: what the sums' loop leaves of the
// registers is too little for more than one way out.)
template <bool kGated, bool kIndex, bool kAligned>
__global__ void __launch_bounds__(Warps<kIndex>::kThreads, 1)
    fp8_matmul_tiles_kernel(const __grid_constant__ MatmulParams p) {
  constexpr int kStages = kStagesOf<kGated, kAligned>;
  extern __shared__ uint8_t raw[];
  PairBlock b;
  b.sm = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  b.base = smem_addr(b.sm);
  b.bars = b.base + kOffBars;
  b.rank = (int)cluster_rank();
  b.first = blockIdx.x / 2;
  b.stride = gridDim.x / 2;
  b.abort = b.bars + kAbort;
  ExpertTiles& tiles = *reinterpret_cast<ExpertTiles*>(b.sm + kOffTiles);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kMostStages; ++i) {
      mbar_init(b.bars + kFull + 8 * i, kIndex ? 3 : 1);
      mbar_init(b.bars + kCopied + 8 * i, 128);
      mbar_init(b.bars + kEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b.bars + kAccFull + 8 * i, 1);
      mbar_init(b.bars + kAccEmpty + 8 * i, 16);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(b.bars + kFactorFull + 8 * i, 2);
      mbar_init(b.bars + kFactorEmpty + 8 * i, 8);
    }
    mbar_init(b.bars + kDrain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
    *reinterpret_cast<volatile int*>(b.sm + kOffBars + kAbort) = 0;
  }
  if (warp == kMmaWarp) pair_alloc(b.bars + kTmemSlot, 512);
  tc_fence_before();
  count_tiles<kTileRows, Warps<kIndex>::kThreads>(p, tiles);
  if (tid == 0) *reinterpret_cast<volatile int*>(b.sm + kOffBars + kTotal) = tiles.tile_start[p.experts];
  __syncthreads();
  // (no data passes with it; at the end arrivals under way do)
  cluster_arrive();
  cluster_wait_all();
  tc_fence_after();
  b.tmem = *reinterpret_cast<volatile uint32_t*>(b.sm + kOffBars + kTmemSlot);
  b.total = tiles.tile_start[p.experts];

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Warps<kIndex>::kSums));
    sum_tiles<kGated, kIndex, kAligned>(p, b.base, b.tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Warps<kIndex>::kOthers));
    if (warp == kLoadWarp) {
      load_tiles<kStages, kGated, kIndex>(p, tiles, b);
    } else if (warp == kMmaWarp) {
      if (b.rank == 0)
        issue_tiles<kStages, kIndex>(p, b);
    } else if (!kIndex || warp < kCopyWarp) {
      serve_factors<kGated>(p, tiles, b);
    } else {
      copy_rows<kStages>(p, tiles, b);
    }
  }
  __syncthreads();
  if (tid == 0 && *reinterpret_cast<volatile int*>(b.sm + kOffBars + kAbort) && p.status)
    atomicExch(p.status, 1);
  cluster_sync();
  if (warp == kMmaWarp) pair_dealloc(b.tmem, 512);
}

template <bool kGated, bool kIndex, bool kAligned>
int launch(const MatmulParams& p, cudaStream_t stream) {
  const auto kernel = fp8_matmul_tiles_kernel<kGated, kIndex, kAligned>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Warps<kIndex>::kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2);
  static int pairs[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
  if (!pairs[dev]) {
    int found = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) != cudaSuccess || found < 1) {
      cudaGetLastError();
      return KVQ_ECUDA;
    }
    pairs[dev] = found;
  }
  const int64_t row_tiles =
      p.offsets ? (int64_t)p.num_rows / kTileRows + (p.num_rows < p.experts ? p.num_rows : p.experts)
                : p.row_tiles_dense;
  const int64_t most = row_tiles * p.column_tiles;
  cfg.gridDim = dim3((unsigned)(2 * (most < pairs[dev] ? most : pairs[dev])));
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  return launch_status();
}

}  // namespace

int launch_matmul_tiles(const MatmulParams& p, bool is_gated, cudaStream_t stream) {
  const bool aligned = p.wide && p.n % 128 == 0;
  if (p.rows)
    return is_gated  ? launch<true, true, true>(p, stream)
           : aligned ? launch<false, true, true>(p, stream)
                     : launch<false, true, false>(p, stream);
  return is_gated  ? launch<true, false, true>(p, stream)
         : aligned ? launch<false, false, true>(p, stream)
                   : launch<false, false, false>(p, stream);
}

}  // namespace kvq
