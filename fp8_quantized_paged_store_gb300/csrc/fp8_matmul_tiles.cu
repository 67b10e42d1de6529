// fp8_matmul_tiles.cu — the kernel of the block-scaled 8-bit products for many
// rows to a matrix.
//
//   out[i][j] = sum_g sa[i][g] sb[j/128][g] sum_{l in g} a[i][l] b[j][l]
//
// A pair of blocks (cta_group::2) takes 256 of b's rows, features, as the M side of
// tcgen05.mma and up to 256 of a's rows as its N side: rows of an expert are
// rounded up to 32, not to a tile. A step is a group of 128 values: each block
// loads 128 features and half of the rows, 32 KB by TMA, for 512 cycles of the
// tensor cores at their rate; four MMAs form the group's product in one of two
// accumulators (256 columns each, all of tensor memory), and eight warps add it,
// scaled, to sums in registers while the next one is formed:
//   acc[t] += partial[t] * (sa[t] sb).
// Accumulators are read in pieces of 16 features x 4 rows: a thread has every
// fourth row, so that a warp reads its factors for 32 features x 32 rows in two
// accesses of 16 bytes (one feature to a thread would take eight), and pieces of
// 8 x 8 transpose on their way through shared memory into out's order.
//
// Gated: a block's 128 features are 64 of a gate block's and the 64 of the up
// half that belong to them. Gate and up warps exchange half of their sums each,
// and the two blocks their largest values, before the codes are formed.
//
// Roles: warps 0-7 sums (lanes of 32 features by warp % 4, half of the rows by
// warp / 4), 8 TMA, 9 MMA (of the first block), 10 and 11 scales. Tiles are
// taken in turn by resident pairs; loads and products run ahead over a tile's end.
#include "fp8_matmul.cuh"
#include "kvq_host.h"

namespace kvq {
namespace {

constexpr int kTileRows = 256;
constexpr int kTileThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kScaleWarp = 10;
// Registers of a thread: 168 at launch, handed to the sums.
constexpr int kSumRegs = 216, kOtherRegs = 72;
static_assert(256 * kSumRegs + 128 * kOtherRegs <= kTileThreads * 168);

template <bool kGated>
struct Tiles {
  static constexpr int kStages = kGated ? 5 : 6;
  static constexpr int kGroup = kGated ? 2 : 4;  // steps whose factors pass together
  static constexpr int kSets = kGated ? 2 : 1;   // of factors: gate's, up's
  static constexpr uint32_t kHalf = 128 * kGroupK;
  static constexpr uint32_t kStageBytes = 2 * kHalf;
  static constexpr uint32_t kFactorBytes = kSets * kTileRows * 4;
  static constexpr uint32_t kWarpBytes = kGated ? 4096 : 1024;  // a sum warp's own
  static constexpr uint32_t kOffFactors = kStages * kStageBytes;
  static constexpr uint32_t kOffWarps = kOffFactors + 2 * kGroup * kFactorBytes;
  // largest values: [tile's parity][block, warp's features][row]
  static constexpr uint32_t kTopBytes = kGated ? 4 * kTileRows * 4 : 0;
  static constexpr uint32_t kOffTops = kOffWarps + 8 * kWarpBytes;
  static constexpr uint32_t kOffTiles = kOffTops + 2 * kTopBytes;
  static constexpr uint32_t kOffBars = (kOffTiles + sizeof(ExpertTiles) + 15) / 16 * 16;
  static constexpr uint32_t kFull = 0, kEmpty = 8 * kStages;
  static constexpr uint32_t kAccFull = 16 * kStages, kAccEmpty = kAccFull + 16;
  static constexpr uint32_t kFactorFull = kAccEmpty + 16, kFactorEmpty = kFactorFull + 16;
  static constexpr uint32_t kTopFull = kFactorEmpty + 16, kDrain = kTopFull + 16;
  static constexpr uint32_t kTmemSlot = kDrain + 8, kAbort = kTmemSlot + 4;
  static_assert(kAbort + 4 <= 512);
  static constexpr size_t kBytes = kOffBars + 512 + 1024;  // room to align the base
  static_assert(kBytes <= 232448);
};

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
__device__ __forceinline__ void pair_gather4(uint32_t dst, const CUtensorMap* map, int x, int y0,
                                             int y1, int y2, int y3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(bar)
      : "memory");
}

// 16 lanes x 64 columns, to be waited for: registers 2 i and 2 i + 1 are column
// 4 i + lane % 4 of lanes lane / 4 and lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_pieces_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 pieces of 16-bit values, transposed: lane 8 j + c gives the place of
// column c of piece j.
__device__ __forceinline__ void st_transposed(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2,
                                              uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// Place of a row's factor: a thread's sixteen of 64 rows, 4 i + q, lie together, four
// at a time, the pairs of fours of q = 2 and 3 the other way round (the four q's
// accesses then meet no bank twice).
__device__ __forceinline__ int factor_place(int row) {
  const int q = row & 3, i = (row & 63) >> 2;
  return (row & ~63) + q * 16 + 4 * ((i >> 2) ^ (q >> 1)) + (i & 3);
}

// Row of the 8 that column c of an 8 x 8 piece stands for: a thread's two columns, 2 q
// and 2 q + 1, hold rows q and q + 4.
__device__ __forceinline__ int piece_row(int c) { return (c >> 1) + 4 * (c & 1); }

struct PairTile {
  int expert, row0, rows, column;
};

__device__ __forceinline__ PairTile pair_tile(const MatmulParams& p, const ExpertTiles& s,
                                              int index) {
  PairTile t;
  t.expert = expert_of_tile(p, s, index);
  const int at = index - s.tile_start[t.expert];
  const int tiles = (s.rows[t.expert] + kTileRows - 1) / kTileRows;
  t.column = at / tiles;
  const int r = at - t.column * tiles;
  t.row0 = s.row_start[t.expert] + r * kTileRows;
  t.rows = min(kTileRows, s.rows[t.expert] - r * kTileRows);
  return t;
}
__device__ __forceinline__ int tile_n(const PairTile& t) { return (t.rows + 31) & ~31; }

struct PairBlock {
  uint8_t* sm;
  uint32_t base, bars, tmem, abort;
  int rank, first, stride, total;
};

template <bool kGated>
__device__ __forceinline__ void load_tiles(const MatmulParams& p, const ExpertTiles& tiles,
                                           const PairBlock& b) {
  using T = Tiles<kGated>;
  const int lane = threadIdx.x & 31;
  uint32_t it = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride) {
    const PairTile t = pair_tile(p, tiles, index);
    const int from = b.rank * (tile_n(t) / 2);  // this block's rows of the tile
    int r[4] = {0, 0, 0, 0};
    if (p.rows) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bool in;
        r[i] = a_row(p, t.row0 + min(from + 4 * lane + i, t.rows - 1), in);
      }
    }
    for (int kb = 0; kb < p.steps; ++kb, ++it) {
      const int st = it % T::kStages;
      if (it >= T::kStages &&
          !uniform_wait(b.bars + T::kEmpty + 8 * st, (it / T::kStages - 1) & 1, b.abort)) {
        ok = false;
        break;
      }
      const uint32_t dst = b.base + st * T::kStageBytes;
      const uint32_t full = in_cluster(b.bars + T::kFull + 8 * st, 0);
      if (lane == 0) {
        if (b.rank == 0) mbar_expect_tx(b.bars + T::kFull + 8 * st, 2 * T::kStageBytes);
        if (kGated) {
          const int y = t.column * 128 + b.rank * 64;
          pair_load_3d(dst, &p.b_map, kb * kGroupK, y, t.expert, full);
          pair_load_3d(dst + T::kHalf / 2, &p.b_map, kb * kGroupK, y + p.up_blocks * 128, t.expert,
                       full);
        } else {
          pair_load_3d(dst, &p.b_map, kb * kGroupK, t.column * 256 + b.rank * 128, t.expert, full);
        }
        if (!p.rows) pair_load_2d(dst + T::kHalf, &p.a_map, kb * kGroupK, t.row0 + from, full);
      }
      __syncwarp();
      if (p.rows)
        pair_gather4(dst + T::kHalf + lane * 4 * kGroupK, &p.a_map, kb * kGroupK, r[0], r[1], r[2],
                     r[3], full);
    }
  }
  // the first block's arrivals here end before this block does
  for (uint32_t i = it > T::kStages ? it - T::kStages : 0; ok && i < it; ++i)
    ok = uniform_wait(b.bars + T::kEmpty + 8 * (i % T::kStages), (i / T::kStages) & 1, b.abort);
  // copies that no MMA will wait for end before the pair does
  if (b.rank == 0 && gone(b.abort)) {
    for (uint32_t i = it > T::kStages ? it - T::kStages : 0; i < it; ++i)
      for (uint32_t n = 0; n < kWaitPolls &&
                           !mbar_test(b.bars + T::kFull + 8 * (i % T::kStages), (i / T::kStages) & 1);)
        ++n;
  }
}

template <bool kGated>
__device__ __forceinline__ void issue_tiles(const MatmulParams& p, const ExpertTiles& tiles,
                                            const PairBlock& b) {
  using T = Tiles<kGated>;
  uint32_t it = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride) {
    const PairTile t = pair_tile(p, tiles, index);
    const uint32_t idesc = instr_desc_f8(256, tile_n(t));
    for (int kb = 0; kb < p.steps; ++kb, ++it) {
      const int st = it % T::kStages, buf = it & 1;
      // (the first use of an accumulator passes: the phase before the first)
      ok = uniform_wait2(b.bars + T::kAccEmpty + 8 * buf, (it / 2 + 1) & 1, b.bars + T::kFull + 8 * st,
                      (it / T::kStages) & 1, b.abort);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = b.base + st * T::kStageBytes;
      const uint64_t features = smem_desc(at, 16, 1024, 2);
      const uint64_t rows = smem_desc(at + T::kHalf, 16, 1024, 2);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          pair_mma(b.tmem + buf * kTileRows, desc_at(features, 32 * j), desc_at(rows, 32 * j), idesc,
                   j > 0);
        pair_commit(b.bars + T::kEmpty + 8 * st);
        pair_commit(b.bars + T::kAccFull + 8 * buf);
      }
      __syncwarp();
    }
  }
  // (bounded, abort or not: no MMA is left when the pair ends)
  if (elect_one())
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            b.bars + T::kDrain)
        : "memory");
  __syncwarp();
  for (uint32_t i = 0; i < kWaitPolls; ++i)
    if (mbar_test(b.bars + T::kDrain, 0)) return;
  give_up(b.abort);
}

// sa[row][g] * sb[g] of 128 rows for every step, a group of steps at a time (a row's
// scales are neighbours in memory), the next group's loads under way.
template <bool kGated>
__device__ __forceinline__ void load_factors(const MatmulParams& p, const ExpertTiles& tiles,
                                             const PairBlock& b) {
  using T = Tiles<kGated>;
  constexpr int kRowsPer = 4, kAhead = T::kGroup;
  const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) - kScaleWarp;
  float* const to = reinterpret_cast<float*>(b.sm + T::kOffFactors) + part * 128;
  const bool vector = p.a_group_step != 0 && p.a_scale_stride % kAhead == 0 &&
                      reinterpret_cast<uintptr_t>(p.a_scales) % (4 * kAhead) == 0;
  uint32_t group = 0;
  bool ok = true;
  for (int index = b.first; ok && index < b.total; index += b.stride) {
    const PairTile t = pair_tile(p, tiles, index);
    const float* sa[kRowsPer];  // null: a row that does not exist
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const int row = part * 128 + lane + 32 * i;
      bool in = row < t.rows;
      const int64_t at = in ? a_row(p, t.row0 + row, in) : 0;
      sa[i] = in ? p.a_scales + at * p.a_scale_stride : nullptr;
    }
    const int block = kGated ? t.column : min(2 * t.column + b.rank, p.blocks - 1);
    const float* sb = p.b_scales + t.expert * p.b_scale_expert_stride + block * p.b_scale_stride;
    const float* sb_up = sb + p.up_blocks * p.b_scale_stride;
    float x[kRowsPer][kAhead], w[T::kSets][kAhead];
    const auto load = [&](int kb) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool have = kb + j < p.steps;
        w[0][j] = have ? ld_f32(sb + kb + j) : 0.0f;
        if (kGated) w[T::kSets - 1][j] = have ? ld_f32(sb_up + kb + j) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) {
        if (vector && kb + kAhead <= p.steps) {
          if constexpr (kAhead == 4) {
            const float4 v = sa[i] ? ld_f4(sa[i] + kb) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            x[i][0] = v.x;
            x[i][1] = v.y;
            x[i][2] = v.z;
            x[i][3] = v.w;
          } else {
            const float2 v = sa[i] ? __ldg(reinterpret_cast<const float2*>(sa[i] + kb)) : make_float2(0.0f, 0.0f);
            x[i][0] = v.x;
            x[i][1] = v.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            x[i][j] = sa[i] && kb + j < p.steps ? ld_f32(sa[i] + (kb + j) * p.a_group_step) : 0.0f;
        }
      }
    };
    load(0);
    for (int kb = 0; kb < p.steps; kb += kAhead, ++group) {
      const int g = group & 1;
      if (group >= 2 && !uniform_wait(b.bars + T::kFactorEmpty + 8 * g, (group / 2 - 1) & 1, b.abort)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int h = 0; h < T::kSets; ++h)
#pragma unroll
          for (int i = 0; i < kRowsPer; ++i)
            to[((g * T::kGroup + j) * T::kSets + h) * kTileRows + factor_place(lane + 32 * i)] = x[i][j] * w[h][j];
      __syncwarp();
      if (lane == 0) mbar_arrive(b.bars + T::kFactorFull + 8 * g);
      if (kb + kAhead < p.steps) load(kb + kAhead);
    }
  }
}

// A tile's steps: acc += partial * factors for the warp's 32 features and, kFirst and
// kSecond, its first and second 64 rows (gated: an up warp begins with its second 64,
// which it finishes, as a gate warp does its first). Everything else is left out of this
// loop, whose registers are all taken: one spilled costs a trip to L2.
template <bool kGated, bool kFirst, bool kSecond>
__device__ __forceinline__ bool sum_steps(const MatmulParams& p, uint32_t base, uint32_t tmem,
                                          uint32_t& it, uint32_t& group, float (&acc)[4][2][16]) {
  using T = Tiles<kGated>;
  const int quarter = threadIdx.x >> 5 & 3, half = threadIdx.x >> 7, up = kGated ? quarter >> 1 : 0;
  const int q = threadIdx.x & 3;
  const uint32_t bars = base + T::kOffBars;
  const uint32_t factors0 =
      base + T::kOffFactors + (uint32_t)(up * kTileRows + half * 128 + 64 * up + 16 * q) * 4;
  const uint32_t from0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128 + 64 * up;
  const uint32_t flip = (uint32_t)(q >> 1) * 16;
  const int to_second = up ? -64 : 64;
#pragma unroll 1
  for (int kb = 0; kb < p.steps; ++kb, ++it) {
    if (kb % T::kGroup == 0 &&
        !uniform_wait(bars + T::kFactorFull + 8 * (group & 1), (group >> 1) & 1, bars + T::kAbort))
      return false;
    if (!uniform_wait(bars + T::kAccFull + 8 * (it & 1), (it / 2) & 1, bars + T::kAbort)) return false;
    tc_fence_after();
    const uint32_t factors =
        factors0 + ((group & 1) * T::kGroup + kb % T::kGroup) * T::kSets * kTileRows * 4;
    const uint32_t from = from0 + (it & 1) * kTileRows;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool some = s == 0 ? kFirst : kSecond;
      const int row = s == 0 ? 0 : to_second;
      uint4 f[4];
      if (some) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = lds_v4_at((factors + 4 * row + 16 * j) ^ flip);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        if (some) {
          tmem_ld_pieces_issue(from + ((uint32_t)(16 * h) << 16) + row, v);
          tmem_ld_wait(v);
        }
        if (s == 1 && h == 1) {
          tc_fence_before();
          __syncwarp();
          if (elect_one()) arrive_pair(in_cluster(bars + T::kAccEmpty + 8 * (it & 1), 0));
        }
        if (some) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint4 g = f[i / 8];
            const uint32_t u = i / 2 % 4 == 0 ? g.x : i / 2 % 4 == 1 ? g.y : i / 2 % 4 == 2 ? g.z : g.w;
            float& a = acc[2 * s + i / 16][h][i % 16];
            a = fmaf(__uint_as_float(v[i]), __uint_as_float(u), a);
          }
        }
      }
    }
    if (kb % T::kGroup == T::kGroup - 1 || kb == p.steps - 1) {
      __syncwarp();
      if (elect_one()) mbar_arrive(bars + T::kFactorEmpty + 8 * (group & 1));
      ++group;
    }
  }
  return true;
}

// The sums of every tile and their way out.
template <bool kGated>
__device__ __forceinline__ void sum_tiles(const MatmulParams& p, const ExpertTiles& tiles,
                                          const PairBlock& b) {
  using T = Tiles<kGated>;
  const int lane = threadIdx.x & 31, q = lane & 3;
  const uint32_t base = b.base, tmem = b.tmem;
  uint32_t it = 0, group = 0;
  int round = 0;
  bool ok = true;  // (a warp that gives up still takes part in the warps' barriers)
#pragma unroll 1
  for (int index = blockIdx.x / 2;
       index < *reinterpret_cast<const volatile int*>(&tiles.tile_start[p.experts]) && (kGated || ok);
       index += gridDim.x / 2, ++round) {
    float acc[4][2][16];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[c][i / 16][i % 16] = 0.0f;
    if (ok) {
      const int rows = pair_tile(p, tiles, index).rows - (threadIdx.x >> 7) * 128;
      const bool up = kGated && (threadIdx.x >> 6 & 1);
      if (__all_sync(0xFFFFFFFFu, rows > 64))
        ok = sum_steps<kGated, true, true>(p, base, tmem, it, group, acc);
      else if (__all_sync(0xFFFFFFFFu, rows <= 0))
        ok = sum_steps<kGated, false, false>(p, base, tmem, it, group, acc);
      else if (kGated && __all_sync(0xFFFFFFFFu, up))
        ok = sum_steps<kGated, false, true>(p, base, tmem, it, group, acc);
      else
        ok = sum_steps<kGated, true, false>(p, base, tmem, it, group, acc);
    }
    const int warp = threadIdx.x >> 5, quarter = warp & 3, half = warp >> 2;
    const int up = kGated ? quarter >> 1 : 0, r0 = half * 128;  // this warp's rows of the tile
    const uint32_t mine = base + T::kOffWarps + warp * T::kWarpBytes;
    const auto chunk = [&](int c) { return r0 + 32 * (kGated ? c ^ (2 * up) : c); };
    const PairTile t = pair_tile(p, tiles, index);
    // rows whose r lies outside a count as zeros
    uint32_t valid[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bool in = chunk(c) + lane < t.rows;
      if (in) a_row(p, t.row0 + chunk(c) + lane, in);
      valid[c] = __ballot_sync(0xFFFFFFFFu, in);
    }
    if constexpr (!kGated) {
      if (!ok) break;
      const int column = t.column * 256 + b.rank * 128 + quarter * 32;  // of the result
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (chunk(c) >= t.rows) break;
#pragma unroll
        for (int pair = 0; pair < 2; ++pair) {  // 16 rows of the result
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = 2 * pair + i;
            const bool in0 = valid[c] >> (8 * m + q) & 1, in1 = valid[c] >> (8 * m + 4 + q) & 1;
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float* a = &acc[c][h][4 * m + k];
                w[2 * h + k] = narrow2_to(in0 ? a[0] : 0.0f, in1 ? a[2] : 0.0f, p.half != 0);
              }
            // lane 8 j + ..: 16 bytes of features 8 j .. of row 8 i + r
            const int r = piece_row(lane & 7), j = lane >> 3;
            st_transposed(mine + (8 * i + r) * 64 + (j ^ (r >> 1 & 3)) * 16, w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * i + (lane >> 2), j = lane & 3;
            const uint4 v = lds_v4_at(mine + r * 64 + (j ^ ((r & 7) >> 1)) * 16);
            const int row = chunk(c) + 16 * pair + r, at = column + 8 * j;
            if (row < t.rows && at < p.n) {
              uint8_t* to = p.out + (int64_t)(t.row0 + row) * p.out_pitch + 2 * (int64_t)at;
              if (p.wide && at + 8 <= p.n) {
                st_v4(to, v);
              } else {
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (at + k < p.n)
                    asm volatile("st.global.u16 [%0], %1;" ::"l"(to + 2 * k),
                                 "h"((uint16_t)(u[k / 2] >> (16 * (k & 1))))
                                 : "memory");
              }
            }
          }
          __syncwarp();
        }
      }
    } else {
      // each warp sends its sums of the 64 rows that its partner finishes
      const int partner = (warp ^ 2);
      const uint32_t theirs = b.base + T::kOffWarps + partner * T::kWarpBytes;
      const int barrier = 1 + (half * 2 + (quarter & 1));
      float most[16];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* a = &acc[c + 2][i / 4][4 * (i % 4)];
          sts_v4(mine + (i * 32 + lane) * 16, make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]),
                                                         __float_as_uint(a[2]), __float_as_uint(a[3])));
        }
        named_barrier(barrier, 64);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = lds_v4_at(theirs + (i * 32 + lane) * 16);
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          const int m = i % 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float& a = acc[c][i / 4][4 * m + k];
            const float other = __uint_as_float(u[k]);
            const float z = gated(up ? other : a, up ? a : other);
            a = valid[c] >> (8 * m + 4 * (k >> 1) + q) & 1 ? z : 0.0f;
          }
        }
        named_barrier(barrier, 64);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = 0.0f;  // (fmaxf leaves NaN out)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              v = fmaxf(v, fmaxf(fabsf(acc[c][h][4 * m + 2 * k]), fabsf(acc[c][h][4 * m + 2 * k + 1])));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            most[8 * c + 2 * m + k] = v;
          }
      }
      // the largest of this warp's 32 features to both blocks
      const uint32_t tops = T::kOffTops + (round & 1) * T::kTopBytes;
      const uint32_t part = tops + (uint32_t)((b.rank * 2 + (quarter & 1)) * kTileRows) * 4;
      if (lane < 8) {
        const uint32_t to = in_cluster(b.base + part, lane >> 2);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              st_cluster(to + (uint32_t)(chunk(c) + 8 * m + 4 * k + q) * 4, most[8 * c + 2 * m + k]);
      }
      __syncwarp();
      if (ok && lane < 2) arrive_cluster(in_cluster(b.bars + T::kTopFull + 8 * (round & 1), lane));
      ok = ok && cluster_wait(b.bars + T::kTopFull + 8 * (round & 1), (round >> 1) & 1, b.abort);
      const int column = t.column * 128 + b.rank * 64 + (quarter & 1) * 32;  // of the result
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int pair = 0; pair < 2; ++pair) {  // 16 rows of the result
          if (!ok || chunk(c) + 16 * pair >= t.rows) break;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = 2 * pair + i, row = chunk(c) + 8 * m + q;  // and row + 4
            float top[2] = {0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const float* v = reinterpret_cast<const float*>(b.sm + tops) + s * kTileRows + row;
              top[0] = fmaxf(top[0], v[0]);
              top[1] = fmaxf(top[1], v[4]);
            }
            const float to0 = code_factor(top[0]), to1 = code_factor(top[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float* a = &acc[c][h][4 * m];
              w[2 * i + h] = cvt_e4m3x2(a[0] * to0, a[1] * to0) | cvt_e4m3x2(a[2] * to1, a[3] * to1) << 16;
            }
            if (b.rank == 0 && (quarter & 1) == 0 && lane < 4) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (row + 4 * k < t.rows)
                  p.out_scales[(int64_t)(t.row0 + row + 4 * k) * p.out_scale_stride + t.column] =
                      code_scale(top[k]);
            }
          }
          // lane 8 j + ..: 16 codes of features 16 (j % 2) .. of row 8 (j / 2) + r,
          // a feature next to the eighth after it
          {
            const int r = piece_row(lane & 7), j = lane >> 3;
            st_transposed(mine + (8 * (j >> 1) + r) * 32 + ((j & 1) ^ (r >> 2)) * 16, w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          const int r = lane >> 1, j = lane & 1;
          const uint4 v = lds_v4_at(mine + r * 32 + (j ^ ((r & 7) >> 2)) * 16);
          const int row = chunk(c) + 16 * pair + r;
          if (row < t.rows)
            st_v4(p.out + (int64_t)(t.row0 + row) * p.out_pitch + column + 16 * j,
                  make_uint4(__byte_perm(v.x, v.y, 0x6420), __byte_perm(v.z, v.w, 0x6420),
                             __byte_perm(v.x, v.y, 0x7531), __byte_perm(v.z, v.w, 0x7531)));
          __syncwarp();
        }
      }
    }
  }
}

template <bool kGated>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp8_matmul_tiles_kernel(const __grid_constant__ MatmulParams p) {
  using T = Tiles<kGated>;
  extern __shared__ uint8_t raw[];
  PairBlock b;
  b.sm = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  b.base = smem_addr(b.sm);
  b.bars = b.base + T::kOffBars;
  b.rank = (int)cluster_rank();
  b.first = blockIdx.x / 2;
  b.stride = gridDim.x / 2;
  b.abort = b.bars + T::kAbort;
  ExpertTiles& tiles = *reinterpret_cast<ExpertTiles*>(b.sm + T::kOffTiles);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(b.bars + T::kFull + 8 * i, 1);
      mbar_init(b.bars + T::kEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b.bars + T::kAccFull + 8 * i, 1);
      mbar_init(b.bars + T::kAccEmpty + 8 * i, 16);
      mbar_init(b.bars + T::kTopFull + 8 * i, 16);
      mbar_init(b.bars + T::kFactorFull + 8 * i, 2);
      mbar_init(b.bars + T::kFactorEmpty + 8 * i, 8);
    }
    mbar_init(b.bars + T::kDrain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
    *reinterpret_cast<volatile int*>(b.sm + T::kOffBars + T::kAbort) = 0;
  }
  if (warp == kMmaWarp) pair_alloc(b.bars + T::kTmemSlot, 2 * kTileRows);
  tc_fence_before();
  count_tiles<kTileRows, kTileThreads>(p, tiles);
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  b.tmem = *reinterpret_cast<volatile uint32_t*>(b.sm + T::kOffBars + T::kTmemSlot);
  b.total = tiles.tile_start[p.experts];

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    sum_tiles<kGated>(p, tiles, b);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      load_tiles<kGated>(p, tiles, b);
    } else if (warp == kMmaWarp) {
      if (b.rank == 0) issue_tiles<kGated>(p, tiles, b);
    } else {
      load_factors<kGated>(p, tiles, b);
    }
  }
  __syncthreads();
  if (tid == 0 && *reinterpret_cast<volatile int*>(b.sm + T::kOffBars + T::kAbort) && p.status)
    atomicExch(p.status, 1);
  cluster_sync();
  if (warp == kMmaWarp) pair_dealloc(b.tmem, 2 * kTileRows);
}

template <bool kGated>
int launch(const MatmulParams& p, cudaStream_t stream) {
  using T = Tiles<kGated>;
  const auto kernel = fp8_matmul_tiles_kernel<kGated>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = T::kBytes;
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
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)T::kBytes) !=
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
  return is_gated ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace kvq
