// fp8_attention.cuh — what the kernels of fp8_paged_attention share: their
// parameters, the masks, and the layout of partial results.
#pragma once

#include "fp8_cache.cuh"

namespace kvq {

// A row keeps two references over the keys that it sees: m, for the scores x_j,
// which the normaliser's sum is relative to, and m + d, for x_j + ev_j (ev: the
// exponent of the page's value scale), which the second product is relative to.
// A product p_j 2**ev_j enters as fp16, times 2**kPLog2. m + d is never above the
// row's largest x_j + ev_j so far, and the row's sums are rescaled before it
// falls kLagLog2 behind: a stored product is at most 2**(9 + 6) < 65504, and
// rounded by more than 2**-11 of itself only below 2**-23 of the row's largest,
// then by at most 2**-34 of that. (With one reference for all rows'
// value scales, a page that a row hardly attends to, or does not see, took the
// other pages' values away from it.)
constexpr float kPLog2 = 9.0f, kLagLog2 = 6.0f;
// A page whose values count for less than 2**-60 of the row's largest product
// still counts fully in the normaliser: the exponent that its products are
// stored with falls no further. m falls at most kScoreLagLog2 behind, so that
// those products, below 2**(20 - 60 + 9), are zeros in fp16.
constexpr float kVFloorLog2 = -60.0f, kScoreLagLog2 = 20.0f;
// Kept instead of m: b = kPLog2 - m, this before the first key (a score of -inf
// then stays one).
constexpr float kNoKey = 3.402823466e38f;

// Rows of a key head up to which a sequence takes the row kernel, in passes of
// 16 over its keys. 64 sequences with 4000 keys in 8 key heads of 128: 16 rows
// 105 us (in the tile kernel 241), 20 rows 178 (241), 32 rows 185 (241); a
// third pass would take longer than the tile kernel, which has room for 256
// rows. Four such sequences: 16 rows 20 us (26), 32 rows 24 (27).
constexpr int kFewRows = 32;
constexpr int kRowTokens = 32;   // keys of one tile of the row kernel
constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;

struct Fp8AttnParams {
  Fp8Cache cache;
  Fp8Seqs seqs;  // lens: keys of each sequence
  const uint8_t* q;
  uint8_t* out;
  float* lse;       // or null
  int32_t* status;  // or null
  int64_t q_token, q_head, o_token, o_head;  // bytes
  int64_t window;   // 0: none
  float scale_log2;  // sm_scale * log2(e)
  int32_t heads, kv_heads, group;
  int32_t causal, half;
  // Row kernel: sequences with 1..row_limit rows (queries x group) each.
  int32_t row_limit;
  int32_t row_tile;        // rows a block has room for (8 or 16)
  int32_t row_grid;        // its blocks
  float* row_partials;     // outputs [row_grid][2][row_tile][head_dim]
  float* row_lse;          // log-sum-exps [row_grid][2][row_tile], log2 units
  // Tile kernel: sequences with more rows than row_limit.
  int64_t tile_units;      // row tiles of 256 a key head has at most, over all sequences
  int32_t tile_chunks;     // parts the keys of a unit are split into at most
  float* tile_partials;    // [tile_units][kv_heads][tile_chunks][256][head_dim + 8]
};

// Tiles of 64 keys a part has at least: a block's start-up and its share of
// the join cost a few tiles' time.
constexpr int kMinChunkTiles = 8;

// A sequence: its rows and how many keys it has. The host keeps every
// sequence's capacity and num_tokens * group below 2**31.
struct SeqSpan {
  int first_row, n, keys;
};

__device__ __forceinline__ SeqSpan seq_span(const Fp8AttnParams& p, int s) {
  int64_t first, n;
  seq_rows(p.seqs, s, first, n);
  SeqSpan r;
  r.first_row = (int)first;
  r.n = (int)n;
  r.keys = (int)clamp64(p.seqs.lens[s], 0, p.cache.capacity);
  return r;
}

// Keys [lo, hi) that some query of [q0, q1) sees.
__device__ __forceinline__ void key_range(const Fp8AttnParams& p, const SeqSpan& s, int q0, int q1,
                                          int& lo, int& hi) {
  hi = p.causal ? max(s.keys - s.n + q1, 0) : s.keys;
  lo = p.window ? (int)clamp64((int64_t)s.keys - s.n + q0 + 1 - p.window, 0, s.keys) : 0;
}

// Place of a row in lse [num_tokens, num_heads], which may have more than 2**31
// of them.
__host__ __device__ constexpr int64_t lse_place(int64_t token, int heads, int head) {
  return token * heads + head;
}
static_assert(lse_place(1 << 20, 4096, 7) == ((int64_t)1 << 32) + 7);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Raises a row's references to cover `top`, the largest score of more keys, and
// `both`, their largest score plus value exponent; the sums so far then take the
// factors f_sum and f_out. A key that raises both is stored as a power of two,
// without rounding: one that takes all the weight gives its value as it is.
// (Rising by whole steps instead, to keep the factors powers of two, cost a
// quarter more error over 16,000 keys.)
__device__ __forceinline__ void raise_refs(float top, float both, float& b, float& d, float& f_sum,
                                           float& f_out) {
  const bool first = b == kNoKey;
  const float step = first ? __int_as_float(0x7F800000) : fmaxf(top + b - kPLog2, 0.0f);
  if (step > 0.0f) b = kPLog2 - top;
  const float to = fmaxf(d - step, both + b - kPLog2);
  f_sum = ex2(-step);
  f_out = ex2(d - to - step);
  d = to;
}

// The square root of 2**x. The parts of a row are weighted by it twice, so that
// one whose probabilities are 2**-200 of the others' still counts when its
// values are as much larger.
__device__ __forceinline__ float root_ex2(float x) { return ex2(0.5f * x); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7F800000); }

// E8M0 byte as a power of two (255: NaN) and as its exponent.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 255u ? __int_as_float(0x7FC00000)
                   : __uint_as_float(b == 0u ? 0x00400000u : b << 23);
}
__device__ __forceinline__ float e8m0_log2(uint32_t b) {
  return b == 255u ? __int_as_float(0x7FC00000) : (float)((int)b - 127);
}

// The row kernel's work: every sequence with 1..row_limit rows to a key head
// has, for each key head, one unit of tiles of 32 keys for each `row_tile`
// rows (next to each other, so that the second finds the keys in L2). All
// units' tiles, in that order, are shared out evenly over `blocks` blocks. The
// host keeps the number of all tiles below 2**32.
struct RowShare {
  SeqSpan span;
  uint32_t tiles;  // of one unit of the sequence
  int rows;        // queries x group, 0: not this kernel's
  int first;       // its first tile
  int units;       // of the sequence
};

static_assert(kFewRows <= 2 * 16, "a sequence has at most two units for a key head");
__device__ __forceinline__ RowShare row_share(const Fp8AttnParams& p, int s) {
  RowShare r;
  r.span = seq_span(p, s);
  r.rows = r.span.n * p.group;
  if (r.rows > p.row_limit) r.rows = 0;
  int lo, hi;
  key_range(p, r.span, 0, r.span.n, lo, hi);
  r.first = lo / kRowTokens;
  r.tiles = r.rows && hi > lo ? (uint32_t)((hi - 1) / kRowTokens + 1 - r.first) : 0u;
  r.units = p.kv_heads * (r.rows > p.row_tile ? 2 : 1);
  return r;
}

// Blocks that take part: every one gets a tile for each of its warps.
__device__ __forceinline__ uint32_t row_blocks(const Fp8AttnParams& p, uint32_t total) {
  const uint32_t most = (total + kRowWarps - 1) / kRowWarps;
  return most < (uint32_t)p.row_grid ? most : (uint32_t)p.row_grid;
}

// First tile of block b's share (the first total % blocks blocks have one tile
// more), and the block that holds a tile.
__device__ __forceinline__ uint32_t share_start(uint32_t b, uint32_t total, uint32_t blocks) {
  const uint32_t per = total / blocks, more = total - per * blocks;
  return b * per + min(b, more);
}
__device__ __forceinline__ uint32_t share_block(uint32_t tile, uint32_t total, uint32_t blocks) {
  const uint32_t per = total / blocks, more = total - per * blocks;
  const uint32_t longer = more * (per + 1);
  return tile < longer ? tile / (per + 1) : more + (tile - longer) / per;
}

}  // namespace kvq
