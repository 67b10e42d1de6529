// fp8_attention_tiles.cu — the tile kernel of fp8_paged_attention: many query
// rows of a key head (prompts, chunks of prompts, wide groups of heads) on
// the tcgen05 tensor cores, and the kernel that joins its partial results.
//
//   x_j = q . k_j * 2**ek(page) * sm_scale,  p_j = 2**(x_j - m),
//   out = sum_j p_j v_j * 2**ev(page) / sum_j p_j
//
// A block takes 256 query rows (queries x the heads of one key head) of a
// sequence as two tiles of 128, and the 64-key tiles that some row sees. E4M3
// codes are exact in fp16, so both products run as kind::f16 with fp16 operands
// and fp32 accumulators. Roles:
//   - producers (warps 8-11 for keys and 12-15 for values, 16 rows of a tile
//     each): codes from the pages into registers two tiles ahead, widened to fp16
//     into 128-byte-swizzled shared memory: keys are read K-major, values
//     MN-major from the same layout (four stages); each also passes its rows'
//     page scales on;
//   - score issuers (warps 16 and 17, one thread each, one for each row tile):
//     S = Q K^T into one of two buffers, once the product of values that reads
//     P from the buffer's columns has completed;
//   - value issuers (warps 18 and 19): O += P V once P has been written over
//     the scores. (One thread for both products of a row tile was the pace: a
//     wait costs it 250 cycles even for a completed barrier.)
//   - softmax (warps 0-3 and 4-7, a row per thread): reads a row's 64 scores
//     into registers, writes P as fp16 pairs over them in tensor memory. With
//     two score buffers the next tile's scores are there when it is done: a
//     product's 200 cycles of latency and the wait for the columns stay off
//     its path.
// The page scales are powers of two. A key's enters with the softmax scale; a
// value's is added to the exponent of the probability that enters the second
// product, relative to the row's own reference, and taken out again of the
// normaliser's sum.
//
// Bound by the chain that a step of 64 keys goes round, not by a rate: 8192
// tokens of 32 heads on 8 key heads of 128 take 482 us (1.14 PFLOP/s, 60 % of
// a plain product's rate), tensor pipe active 49 % of the time, issue slots 60
// %. A step takes 1,900 cycles: the softmax of a row's 64 scores 1,400 from one
// look at a barrier to the next, the two products 1,300 on the tensor pipe, and
// every notice between them 250 to 500. Tried and slower: two threads a row (24
// warps), scores loaded ahead, one score buffer with the probabilities apart,
// arrivals by warps. A block's start and end cost 11 steps' time.
//
// The stages leave next to no L1, so a spilled register costs a trip to L2:
// the loops are written to need none (with 300 bytes spilled a tile took twice
// as long), and kept small for the instruction caches (twice the code: the
// same).
//
// Few row tiles (a chunk behind a long context) are split over the keys as
// well, so that the grid fills the SMs; a second kernel joins the parts.
#include "fp8_attention.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTileM = 128;  // rows of a tile
constexpr int kTileK = 64;   // keys of a tile
constexpr int kTileThreads = 640;
constexpr int kProducerWarp = 8, kScoreWarp = 16, kValueWarp = 18;
// Registers of a thread: 96 at launch, then handed from the other roles to the
// softmax (256 x 144 + 256 x 80 + 128 x 32 of 640 x 96). With 128 for the
// softmax a prompt of 8192 tokens took 567 us, with 144 525.
constexpr int kSoftmaxRegs = 144, kProducerRegs = 80, kIssuerRegs = 32;
constexpr int kBlockRegs = 256 * kSoftmaxRegs + 256 * kProducerRegs + 128 * kIssuerRegs;
static_assert(kBlockRegs <= kTileThreads * 96);
constexpr int kKvStages = 4;

// The page scales of a tile, by 16 keys.
struct TileMeta {
  float4 k_scale;  // 2**ek
  float4 v_log2;   // ev, -inf without a page
};

// mbarriers (byte offsets): kKvStages each, then two for each row tile (row
// tile c, buffer b at 16 c + 8 b)
constexpr uint32_t kKFull = 0, kVFull = 32, kEmpty = 64, kMetaFull = 96;
constexpr uint32_t kSFull = 128, kPFull = 160, kPvDone = 192;
constexpr uint32_t kDrain = 224;  // one for each issuer
constexpr uint32_t kTmemSlot = 256, kAbort = 260, kNanMask = 264, kBarBytes = 272;

__device__ __forceinline__ void sts_v2(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ int2 lds_int2(uint32_t a) {
  int2 v;
  asm volatile("ld.shared.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Both barriers' phases; tested together, so that the second adds no latency.
__device__ __forceinline__ bool mbar_wait2(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb,
                                           volatile int* abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    const bool da = mbar_test(a, pa), db = mbar_test(b, pb);
    if (da && db) return true;
    if ((i & 31u) == 31u && *abort) return false;
  }
  *abort = 1;
  return false;
}

// Largest of three, NaN if any is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void tmem_st16_issue(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 codes where `have`, else zeros; issued where it stands.
__device__ __forceinline__ uint4 ld_codes(const uint8_t* p, bool have) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"((uint32_t)have));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Bit 7 of a byte is set where the code is the E4M3 NaN (other bits: anything).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return (w & 0x7F7F7F7Fu) + 0x01010101u;
}

// Keeps the compiler from peeling a loop's first turns, or from copying the
// loop for each value of a condition (the kernel's code has to stay small: at
// twice the size, instruction fetches took most of the time).
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// Floats of a partial row: its elements, its log-sum-exp, and room to a
// multiple of 32 bytes.
template <int kD>
constexpr int64_t kPartPitch = kD + 8;

// 32 aligned bytes: half the passes of two stores of 16 when the lanes' rows
// lie apart.
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A block's work: rows [row0, row0 + rows) of the unit (sequence, key head),
// against key tiles [t0, t1).
struct TileWork {
  SeqSpan span;
  int row0, rows;
  int q0, h0;            // query and head (of the group) of the first row
  int u0, u1;            // all tiles of the unit
  int t0, t1;            // this block's
  int all_lim, all_low;  // keys in [all_low, all_lim) are seen by every row
  int chunks;            // non-empty parts of the unit
  int seq, head;
  uint32_t part;         // place of this block's partial result
};

__device__ __forceinline__ uint32_t tile_units(const Fp8AttnParams& p, const SeqSpan& span) {
  const int rows = span.n * p.group;
  return rows > p.row_limit ? (uint32_t)(rows + 2 * kTileM - 1) / (2 * kTileM) : 0u;
}

// The sequence that the y-th of all units belongs to, and the units before its
// first. Longest sequence first, so that the last blocks to start are short
// ones (six chunks behind contexts of 1,300 to 12,000 tokens took 600 us in the
// batch's order and 522 us so). With more than kSorted sequences: from the last
// to the first. Called by a whole block.
constexpr int kSorted = 256;
template <int kThreads>
__device__ __forceinline__ bool find_unit(const Fp8AttnParams& p, uint32_t y, int& seq,
                                          uint32_t& before) {
  const int count = p.seqs.count;
  if (count > kSorted) {
    uint32_t total;
    const auto reversed = [&](int i) -> uint32_t {
      return tile_units(p, seq_span(p, count - 1 - i));
    };
    const bool found = find_share<kThreads>(count, reversed, [&](uint32_t) { return y; }, seq,
                                            before, total);
    seq = count - 1 - seq;
    return found;
  }
  static_assert(kThreads >= kSorted);
  __shared__ int keys_of[kSorted];
  __shared__ uint32_t units_of[kSorted], found_before;
  __shared__ int found_seq;
  const int i = threadIdx.x;
  int keys = 0;
  uint32_t units = 0;
  if (i < count) {
    const SeqSpan span = seq_span(p, i);
    keys_of[i] = keys = span.keys;
    units_of[i] = units = tile_units(p, span);
  }
  if (i == 0) found_seq = -1;
  __syncthreads();
  if (units > 0) {
    uint32_t at = 0;
#pragma unroll 1
    for (int k = 0; k < count; ++k)
      if (keys_of[k] > keys || (keys_of[k] == keys && k < i)) at += units_of[k];
    if (y >= at && y - at < units) {
      found_seq = i;
      found_before = at;
    }
  }
  __syncthreads();
  seq = found_seq;
  before = found_before;
  return seq >= 0;
}

// The `unit`-th row tile pair of the sequence, from its last on.
__device__ __forceinline__ TileWork tile_work(const Fp8AttnParams& p, int s, int unit, int chunk) {
  TileWork w;
  w.span = seq_span(p, s);
  w.row0 = ((int)tile_units(p, w.span) - 1 - unit) * 2 * kTileM;
  w.rows = min(2 * kTileM, w.span.n * p.group - w.row0);
  w.q0 = (int)((uint32_t)w.row0 / (uint32_t)p.group);
  w.h0 = w.row0 - w.q0 * p.group;
  const int q1 = (int)((uint32_t)(w.row0 + w.rows - 1) / (uint32_t)p.group);
  int lo, hi, unused;
  key_range(p, w.span, w.q0, q1 + 1, lo, hi);
  key_range(p, w.span, w.q0, w.q0 + 1, unused, w.all_lim);
  key_range(p, w.span, q1, q1 + 1, w.all_low, unused);
  w.u0 = lo / kTileK;
  w.u1 = hi > lo ? (hi - 1) / kTileK + 1 : w.u0;
  int per = (int)((uint32_t)(w.u1 - w.u0 + p.tile_chunks - 1) / (uint32_t)p.tile_chunks);
  if (per < kMinChunkTiles) per = kMinChunkTiles;
  w.chunks = (int)((uint32_t)(w.u1 - w.u0 + per - 1) / (uint32_t)per);
  w.seq = s;
  w.t0 = min(w.u0 + chunk * per, w.u1);
  w.t1 = min(w.t0 + per, w.u1);
  return w;
}

// Of 32 keys, those that a row sees: [low, lim), and of the two groups of 16
// those with a page (bits of `ok`).
__device__ __forceinline__ uint32_t visible(int lim, int low, uint32_t ok) {
  const int to = min(max(lim, 0), 32), from = min(max(low, 0), 32);
  const uint32_t upto = to < 32 ? (1u << to) - 1u : 0xFFFFFFFFu;
  const uint32_t below = from < 32 ? (1u << from) - 1u : 0xFFFFFFFFu;
  const uint32_t pages = (ok & 1u ? 0xFFFFu : 0u) | (ok & 2u ? 0xFFFF0000u : 0u);
  return upto & ~below & pages;
}

// What belongs to the 16 keys 32 q + 16 g of a tile with kG groups (q is not
// known at compile time).
template <int kG>
__device__ __forceinline__ float of_group(const float (&x)[kG], int q, int g) {
  if constexpr (kG == 1) return x[0];
  if constexpr (kG == 2) return q ? x[1] : x[0];
  if constexpr (kG == 4) return q ? x[2 + g] : x[g];
}

// Query (of the sequence) and head (of the group) of row r of the block.
__device__ __forceinline__ void row_place(const Fp8AttnParams& p, const TileWork& w, int r, int& qi,
                                          int& h) {
  const int at = w.h0 + r;
  const int dq = (int)((uint32_t)at / (uint32_t)p.group);
  qi = w.q0 + dq;
  h = at - dq * p.group;
}

// Whether a value that the row sees among the tile's keys is NaN in elements
// [d, d + 16): a rare path, straight from the cache.
__device__ __noinline__ uint32_t nan_elements(const Fp8AttnParams& p, int s, int head, int key0,
                                              int low, int lim, int d) {
  uint32_t bad = 0;
#pragma unroll 1
  for (int key = max(key0, low); key < min(key0 + kTileK, lim); ++key) {
    const int64_t g = page_of(p.cache, s, key);
    if (g < 0) continue;
    if (p.cache.v_scales[g * p.cache.scale_page_stride + head] == 255) return 0xFFFFFFFFu;
    const uint8_t* row = p.cache.v + g * p.cache.page_stride + head * p.cache.head_stride +
                         (int64_t)(key & ((1 << p.cache.page_log2) - 1)) * p.cache.slot_stride + d;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) bad |= (row[i] & 0x7F) == 0x7F ? 1u << i : 0u;
  }
  return bad;
}

template <int kD>
struct Layout {
  static constexpr uint32_t kBlocks = kD / 64;                  // K-blocks of 64 elements
  static constexpr uint32_t kQBlock = 2 * kTileM * 128;         // 256 rows of 128 bytes
  static constexpr uint32_t kKvBlock = kTileK * 128;
  static constexpr uint32_t kStage = kBlocks * kKvBlock;
  static constexpr uint32_t kOffK = kBlocks * kQBlock;
  static constexpr uint32_t kOffV = kOffK + kKvStages * kStage;
  static constexpr uint32_t kOffMeta = kOffV + kKvStages * kStage;
  static constexpr uint32_t kOffQs = kOffMeta + kKvStages * sizeof(TileMeta);
  static constexpr uint32_t kOffSees = kOffQs + 2 * kTileM * 4;
  static constexpr uint32_t kOffBar = kOffSees + 2 * kTileM * 8;
  static constexpr uint32_t kOffWork = kOffBar + kBarBytes;
  static constexpr uint32_t kOffEnd = kOffWork + 80;
  static constexpr size_t kBytes = kOffEnd + 1024;  // room to align the base
  static constexpr uint32_t kIdescQk = instr_desc(kTileM, kTileK, false, false);
  static constexpr uint32_t kIdescPv = instr_desc(kTileM, kD, true, false);
};
static_assert(sizeof(TileWork) <= 80, "TileWork grew past its place");

// ---------------------------------------------------------------- producer ---

// A page of the block table, and whether it is one.
__device__ __forceinline__ int64_t table_page(const Fp8AttnParams& p, const int64_t* table,
                                              int token, bool have) {
  const int64_t g = have ? table[token >> p.cache.page_log2] : -1;
  return (uint64_t)g < (uint64_t)p.cache.num_pages ? g : -1;
}

// A warp's 16 rows of a tile.
template <int kD>
struct Producer {
  static constexpr int kPieces = kD / 16;           // 16-byte pieces of a row
  static constexpr int kRowsAtOnce = 32 / kPieces;  // rows that a warp's 32 pieces cover
  static constexpr int kLoads = 16 / kRowsAtOnce;

  // The row (of a round) and the piece of a lane. Eight lanes, a store phase,
  // hold two rows' pieces of one 64-element block: their swizzled chunks lie
  // in different banks.
  static __device__ __forceinline__ int row_of(int lane) {
    return kPieces == 8 ? (lane >> 2) & 3 : lane >> 2;
  }
  static __device__ __forceinline__ int piece_of(int lane) {
    return kPieces == 8 ? ((lane >> 4) << 2) + (lane & 3) : lane & 3;
  }

  // Rows i * kRowsAtOnce + the lane's own; `from`: the lane's piece of the
  // first, or null without a page; `left`: tokens from the lane's first row to
  // the sequence's end. Rows past it are zeros, like those without a page.
  static __device__ __forceinline__ void load(const uint8_t* from, int64_t step, int left,
                                              uint4 (&out)[kLoads]) {
    const bool have = from != nullptr;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      out[i] = ld_codes(from, have && i * kRowsAtOnce < left);
      from += step;
    }
  }

  // The same when every row is there.
  static __device__ __forceinline__ void load_all(const uint8_t* from, int64_t step,
                                                  uint4 (&out)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(out[i].x), "=r"(out[i].y), "=r"(out[i].z), "=r"(out[i].w)
                   : "l"(from));
      from += step;
    }
  }

  // The codes as fp16 into a stage, 16 codes as two 16-byte chunks of a
  // swizzled row. `at`: the lane's row of the first round; `even`, `odd`: its
  // first chunk's offset in the rounds of either parity (the second is 16 on
  // or back).
  static __device__ __forceinline__ void store(uint32_t at, uint32_t even, uint32_t odd,
                                               const uint4 (&c)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint4 a, b;
      e4m3x4_to_f16x4(c[i].x, a.x, a.y);
      e4m3x4_to_f16x4(c[i].y, a.z, a.w);
      e4m3x4_to_f16x4(c[i].z, b.x, b.y);
      e4m3x4_to_f16x4(c[i].w, b.z, b.w);
      const uint32_t chunk = i & 1 ? odd : even;
      sts_v4(at + i * (kRowsAtOnce * 128) + chunk, a);
      sts_v4(at + i * (kRowsAtOnce * 128) + (chunk ^ 16u), b);
    }
  }

  // A tile that some row does not see whole: 0 * NaN is NaN, so a NaN that not
  // every row sees is kept out of the product, and the rows that see it are
  // told at the end, by a bit of nan_mask for the tile: counted from the unit's
  // first tile at the lower edge, from its last at the upper (a block's rows
  // span at most 256 queries, so each edge has few such tiles). A page whose
  // value scale is NaN (`bad`) holds NaN.
  static __device__ __forceinline__ void mend(uint4 (&c)[kLoads], bool bad, int left, bool partial,
                                              int from_low, int from_high,
                                              unsigned long long* nan_mask) {
    bool found = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t x[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (bad && i * kRowsAtOnce < left) x[k] = 0x7F7F7F7Fu;
        const uint32_t n = nan_codes(x[k]) & 0x80808080u;
        found |= n != 0u;
        if (partial) x[k] &= ~((n >> 7) * 0xFFu);
      }
      c[i] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    if (found && partial) {
      if (from_low < 32) atomicOr(nan_mask, 1ull << from_low);
      else if (from_high < 32) atomicOr(nan_mask, 1ull << (32 + from_high));
    }
  }
};

// ------------------------------------------------------------------ kernel ---

// kG: groups of keys in a tile that have a page each (1 for pages of 64 or
// more, 2 of 32, 4 of 16).
template <int kD, int kG>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp8_attention_tiles_kernel(const __grid_constant__ Fp8AttnParams p) {
  using L = Layout<kD>;
  using P = Producer<kD>;
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float ninf = neg_inf();

  // this block's unit: a sequence's row tiles from the last to the first (under
  // a causal mask the longest first), and for each its key heads and parts
  const uint32_t wide = (uint32_t)p.kv_heads * (uint32_t)p.tile_chunks;
  const uint32_t y = blockIdx.x / wide;
  const uint32_t x = blockIdx.x - y * wide;
  const int head = (int)(x / (uint32_t)p.tile_chunks);
  const int chunk = (int)(x - (uint32_t)head * (uint32_t)p.tile_chunks);
  int seq;
  uint32_t before;
  if (!find_unit<kTileThreads>(p, y, seq, before)) return;
  TileWork w = tile_work(p, seq, (int)(y - before), chunk);
  w.head = head;
  w.part = (y * (uint32_t)p.kv_heads + (uint32_t)head) * (uint32_t)p.tile_chunks + (uint32_t)chunk;
  const bool half = p.half != 0;

  if (w.t0 >= w.t1) {
    // no keys at all: zeros (one of the unit's blocks writes them)
    if (chunk == 0)
#pragma unroll 1
      for (int id = tid; id < w.rows * (kD / 8); id += kTileThreads) {
        const int r = id / (kD / 8), c = id - r * (kD / 8);
        int qi, h;
        row_place(p, w, r, qi, h);
        h += head * p.group;
        st_v4(p.out + (w.span.first_row + qi) * p.o_token + h * p.o_head + 16 * c,
              make_uint4(0, 0, 0, 0));
        if (c == 0 && p.lse) p.lse[lse_place(w.span.first_row + qi, p.heads, h)] = ninf;
      }
    return;
  }
  const int n_tiles = w.t1 - w.t0;
  const bool two = w.rows > kTileM;  // both row tiles in use

  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const uint32_t bars = base + L::kOffBar;
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kOffBar + kAbort);
  unsigned long long* nan_mask =
      reinterpret_cast<unsigned long long*>(sm + L::kOffBar + kNanMask);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kOffBar + kTmemSlot);
  float* q_scale = reinterpret_cast<float*>(sm + L::kOffQs);
  TileMeta* meta = reinterpret_cast<TileMeta*>(sm + L::kOffMeta);
  TileWork* work = reinterpret_cast<TileWork*>(sm + L::kOffWork);

  if (warp == kScoreWarp) tmem_alloc(smem_addr(tmem_slot), 512);
  if (tid == 32 * kProducerWarp) {
    *work = w;  // for the end, where it is read again
    const uint32_t chains = two ? 2 : 1;
#pragma unroll 1
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(bars + kKFull + 8 * i, 128);
      mbar_init(bars + kVFull + 8 * i, 128);
      mbar_init(bars + kEmpty + 8 * i, chains);
      mbar_init(bars + kMetaFull + 8 * i, 8);
      mbar_init(bars + kSFull + 8 * i, 1);
      mbar_init(bars + kPFull + 8 * i, 128);
      mbar_init(bars + kPvDone + 8 * i, 1);
      mbar_init(bars + kDrain + 8 * i, 1);
    }
    *abort = 0;
    *nan_mask = 0ull;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // producers start their first loads while the softmax warps bring in Q
  const bool producer = warp >= kProducerWarp && warp < kScoreWarp;
  const int prow = 16 * (warp & 3) + P::row_of(lane), piece = P::piece_of(lane);
  const int64_t p_off = head * p.cache.head_stride +
                        (int64_t)P::row_of(lane) * p.cache.slot_stride + 16 * piece;
  const int64_t p_step = (int64_t)P::kRowsAtOnce * p.cache.slot_stride;
  const int64_t* table = p.cache.table + seq * p.cache.table_stride;
  const int keys = w.span.keys;
  // byte offset of the lane's piece of its first row of a tile, -1: no page
  const auto place = [&](int64_t g, int tile) -> int64_t {
    // (slots below 256, their stride at most 2**22)
    const uint32_t slot = (uint32_t)(tile * kTileK + 16 * (warp & 3)) &
                          ((1u << p.cache.page_log2) - 1u);
    return g < 0 ? -1 : g * p.cache.page_stride + slot * (uint32_t)p.cache.slot_stride;
  };
  const auto page_at = [&](int tile) -> int64_t {
    const int token = tile * kTileK + 16 * (warp & 3);
    return table_page(p, table, token, tile < w.t1 && token < keys);
  };
  const bool of_keys = warp < kProducerWarp + 4;
  const uint8_t* codes = (of_keys ? p.cache.k : p.cache.v) + p_off;
  const uint8_t* head_scales = (of_keys ? p.cache.k_scales : p.cache.v_scales) + head;
  uint4 buf[2][P::kLoads];   // this tile's codes and the next one's
  uint32_t byte[2];          // their pages' scales
  bool paged[2];             // and whether there are pages
  int64_t pg_ahead = -1;     // the page of the tile after those
  const auto fetch = [&](int64_t pg, int tile, uint4 (&to)[P::kLoads], uint32_t& scale,
                         bool& have) {
    const int64_t at = place(pg, tile);
    const int left = keys - tile * kTileK;
    if (at >= 0 && left >= kTileK)  // (the usual case, without a test for each row)
      P::load_all(codes + at, p_step, to);
    else
      P::load(at < 0 ? nullptr : codes + at, p_step, left - prow, to);
    have = pg >= 0;
    scale = 127u;
    if (have) scale = ld_u8(head_scales + pg * p.cache.scale_page_stride);
  };
  if (producer) {
    const int64_t pg0 = page_at(w.t0), pg1 = page_at(w.t0 + 1);
    pg_ahead = page_at(w.t0 + 2);
    fetch(pg0, w.t0, buf[0], byte[0], paged[0]);
    fetch(pg1, w.t0 + 1, buf[1], byte[1], paged[1]);
  } else {
    // rows as fp16, each times a power of two that brings its largest
    // magnitude to [2**14, 2**15); 8 threads to a row, a 16-byte piece of each
    // 64 elements each
    constexpr int kAtOnce = (kTileThreads - 256) / 8, kBatch = 3;
    const int id = warp < kProducerWarp ? tid : tid - 256;
    const int c = id & 7;
    // query and head of the thread's next row
    int r = id >> 3, qi, h;
    row_place(p, w, r, qi, h);
    const int q_step = (int)((uint32_t)kAtOnce / (uint32_t)p.group);
    const int h_step = kAtOnce - q_step * p.group;
    const uint8_t* from = p.q + w.span.first_row * p.q_token + head * p.group * p.q_head + 16 * c;
#pragma unroll 1
    for (; r < 2 * kTileM; r += kAtOnce * kBatch) {
      uint4 v[kBatch][L::kBlocks];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const uint8_t* row = from + qi * p.q_token + h * p.q_head;
#pragma unroll
        for (int i = 0; i < (int)L::kBlocks; ++i) {
          v[b][i] = make_uint4(0, 0, 0, 0);
          if (r + b * kAtOnce < w.rows) v[b][i] = ld_once_v4(row + 128 * i);
        }
        qi += q_step;
        h += h_step;
        if (h >= p.group) {
          h -= p.group;
          ++qi;
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        // largest magnitude, by the bits of the 16-bit values
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < (int)L::kBlocks; ++i) {
          const uint4 x = v[b][i];
          top = max_u16x2(top, max_u16x2(max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                         max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
          top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float amax = widen2(max(top & 0xFFFFu, top >> 16), half).x;
        const int e = amax > 0.0f ? max((int)(__float_as_uint(amax) >> 23), 16) - 127 : 0;
        const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
        const int at_row = r + b * kAtOnce;
        if (at_row < 2 * kTileM) {
          if (c == 0)
            q_scale[at_row] = p.scale_log2 * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
          const uint32_t at = base + (uint32_t)at_row * 128 + (((uint32_t)c ^ ((uint32_t)at_row & 7)) << 4);
#pragma unroll
          for (int i = 0; i < (int)L::kBlocks; ++i) {
            float f[8];
            widen8(v[b][i], half, f);
            sts_v4(at + i * L::kQBlock,
                   make_uint4(pack_f16(f[0] * up, f[1] * up), pack_f16(f[2] * up, f[3] * up),
                              pack_f16(f[4] * up, f[5] * up), pack_f16(f[6] * up, f[7] * up)));
          }
        }
      }
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const volatile TileWork& vw = *work;  // what is needed late
  constexpr uint32_t kColO = 256;

  if (producer) {
    // ------------------------------------------------------------ producers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    const uint32_t row_at = base + (of_keys ? L::kOffK : L::kOffV) +
                            (uint32_t)(piece >> 2) * L::kKvBlock + (uint32_t)prow * 128;
    const uint32_t even = ((2u * (uint32_t)(piece & 3)) ^ ((uint32_t)prow & 7u)) << 4;
    const uint32_t odd = even ^ (P::kRowsAtOnce == 4 ? 64u : 0u);
    const uint32_t full = bars + (of_keys ? kKFull : kVFull);
    const auto turn = [&](int j, uint4 (&b)[P::kLoads], uint32_t& scale, bool& have) -> bool {
      const int tile = w.t0 + j, key0 = tile * kTileK;
      const uint32_t st = (uint32_t)(j & (kKvStages - 1));
      const int64_t pg_after = page_at(tile + 3);
      if (!of_keys) {
        const bool bad = scale == 255u;
        const bool partial = key0 + kTileK > w.all_lim || key0 < w.all_low;
        if (bad || partial)
          P::mend(b, bad, keys - key0 - prow, partial, tile - vw.u0, vw.u1 - 1 - tile, nan_mask);
      }
      // (at first the wait for parity 1 passes at once)
      if (!warp_wait(bars + kEmpty + 8 * st, (uint32_t)((j / kKvStages - 1) & 1), abort))
        return false;
      if (lane == 0) {
        // (a value scale that is NaN: see mend)
        TileMeta& m = meta[st];
        if (of_keys)
          (&m.k_scale.x)[warp & 3] = e8m0_value(scale);
        else
          (&m.v_log2.x)[warp & 3] = !have ? ninf : (scale == 255u ? 0.0f : e8m0_log2(scale));
        mbar_arrive(bars + kMetaFull + 8 * st);
      }
      P::store(row_at + st * L::kStage, even, odd, b);
      fence_proxy_async();
      mbar_arrive(full + 8 * st);
      fetch(pg_ahead, tile + 2, b, scale, have);
      pg_ahead = pg_after;
      return true;
    };
#pragma unroll 1
    for (int j = 0; j < n_tiles; j += 2) {
      if (!turn(j, buf[0], byte[0], paged[0])) break;
      if (j + 1 < n_tiles && !turn(j + 1, buf[1], byte[1], paged[1])) break;
    }
  } else if (warp >= kScoreWarp) {
    // -------------------------------------------------------------- issuers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
    const uint32_t c = (uint32_t)(warp & 1);  // row tile
    if (lane == 0 && (c == 0 || two)) {
      const uint32_t s_col = tmem + c * 128;
      const uint32_t s_bar = bars + kSFull + 16 * c, p_bar = bars + kPFull + 16 * c;
      const uint32_t done_bar = bars + kPvDone + 16 * c;
      if (warp < kValueWarp) {
        const uint64_t q_desc = smem_desc(base + c * (kTileM * 128), 16, 1024, 2);
        const uint64_t k_desc0 = smem_desc(base + L::kOffK, 16, 1024, 2);
#pragma unroll 1
        for (int j = 0; j < n_tiles; ++j) {
          const uint32_t st = (uint32_t)(j & (kKvStages - 1)), buf = (uint32_t)(j & 1);
          // (for a buffer's first tile the wait for parity 1 passes at once)
          if (!mbar_wait2(bars + kKFull + 8 * st, (uint32_t)((j / kKvStages) & 1),
                          done_bar + 8 * buf, (uint32_t)(((j >> 1) - 1) & 1), abort))
            break;
          tc_fence_after();
          const uint64_t k_desc = desc_at(k_desc0, st * L::kStage);
#pragma unroll
          for (uint32_t b = 0; b < L::kBlocks; ++b)
#pragma unroll
            for (uint32_t ks = 0; ks < 4; ++ks)
              mma_ss(s_col + 64 * buf, desc_at(q_desc, b * L::kQBlock + ks * 32),
                     desc_at(k_desc, b * L::kKvBlock + ks * 32), L::kIdescQk, (b | ks) != 0);
          mma_commit(s_bar + 8 * buf);
        }
      } else {
        const uint64_t v_desc0 = smem_desc(base + L::kOffV, L::kKvBlock, 1024, 2);
        const uint32_t o_col = tmem + kColO + c * kD;
#pragma unroll 1
        for (int j = 0; j < n_tiles; ++j) {
          const uint32_t st = (uint32_t)(j & (kKvStages - 1)), buf = (uint32_t)(j & 1);
          if (!mbar_wait2(bars + kVFull + 8 * st, (uint32_t)((j / kKvStages) & 1),
                          p_bar + 8 * buf, (uint32_t)((j >> 1) & 1), abort))
            break;
          tc_fence_after();
          const uint64_t v_desc = desc_at(v_desc0, st * L::kStage);
#pragma unroll
          for (uint32_t ks = 0; ks < kTileK / 16; ++ks)
            mma_ts(o_col, s_col + 64 * buf + 8 * ks, desc_at(v_desc, ks * 2048), L::kIdescPv,
                   j != 0 || ks != 0);
          mma_commit(done_bar + 8 * buf);
          // (the tile's scores were complete before P was written)
          mma_commit(bars + kEmpty + 8 * st);
        }
      }
      if (!drain_mmas(bars + kDrain + 8 * (uint32_t)(warp - kScoreWarp))) *abort = 1;
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if (warp < 4 || two) {
      const uint32_t c = (uint32_t)(warp >> 2);
      const int r = tid;  // row of the block
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t o_col = tmem + lanes + kColO + c * kD;
      const float qs = q_scale[r];
      // keys the row sees, from the block's first tile on: in shared memory, for
      // the tiles that not every row of the warp sees whole
      int warp_lim, warp_low;
      {
        int lim = 0x7FFFFFFF, low = 0;
        if (r < w.rows) {
          int qi, h, lo, hi;
          row_place(p, w, r, qi, h);
          key_range(p, w.span, qi, qi + 1, lo, hi);
          lim = hi - w.t0 * kTileK;
          low = lo - w.t0 * kTileK;
        }
        sts_v2(base + L::kOffSees + 8 * r, (uint32_t)lim, (uint32_t)low);
        warp_lim = __reduce_min_sync(0xFFFFFFFFu, lim);
        warp_low = __reduce_max_sync(0xFFFFFFFFu, low);
      }
      float b = kNoKey, d = 0.0f, l = 0.0f;
      bool live = true;
#pragma unroll 1
      for (int j = 0; j < n_tiles; ++j) {
        const uint32_t st = (uint32_t)(j & (kKvStages - 1)), buf = (uint32_t)(j & 1);
        const uint32_t s_col = tmem + lanes + c * 128 + 64 * buf;
        live = __all_sync(0xFFFFFFFFu,
                          mbar_wait2(bars + kMetaFull + 8 * st, (uint32_t)((j / kKvStages) & 1),
                                     bars + kSFull + 16 * c + 8 * buf, (uint32_t)((j >> 1) & 1),
                                     abort));
        if (!live) break;
        tc_fence_after();
        const TileMeta mt = meta[st];
        constexpr int kN = kTileK / kG;  // keys of a group
        float k_scale[kG], ve[kG];
        uint32_t oks = 0;  // of 16 keys, those with a page
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          k_scale[g] = qs * (&mt.k_scale.x)[4 / kG * g];
          ve[g] = (&mt.v_log2.x)[4 / kG * g];
          if (ve[g] != ninf) oks |= ((1u << 4 / kG) - 1u) << (4 / kG * g);
        }
        const int key0 = j * kTileK;
        bool masked = key0 + kTileK > warp_lim || key0 < warp_low || oks != 15u;
        float top = ninf, both = ninf;  // largest score; plus value exponent
        uint32_t a[2][32];
        if (!masked) {
          tmem_ld32_issue(s_col, a[0]);
          tmem_ld32_issue(s_col + 32, a[1]);
          tmem_ld_wait(a[0]);
          after_wait(a[1]);
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const auto x = [&](int k) { return __uint_as_float(a[(kN * g + k) >> 5][(kN * g + k) & 31]); };
            float mx[2] = {x(0), x(1)};
#pragma unroll
            for (int k = 2; k < kN - 2; k += 4) {
              mx[0] = max3_nan(mx[0], x(k), x(k + 1));
              mx[1] = max3_nan(mx[1], x(k + 2), x(k + 3));
            }
            mx[0] = max3_nan(mx[0], x(kN - 2), x(kN - 1));
            const float of_g = fmaxf(mx[0], mx[1]) * k_scale[g];
            top = max3_nan(top, mx[0] * k_scale[g], mx[1] * k_scale[g]);
            both = fmaxf(both, of_g + ve[g]);
          }
          // (a NaN score leaves the references to the general path)
          if (__any_sync(0xFFFFFFFFu, top != top)) {
            masked = true;
            top = both = ninf;
          }
        }
        if (masked) {
          const int2 sees = lds_int2(base + L::kOffSees + 8 * r);
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t x[32];
            tmem_ld32_issue(s_col + 32 * q, x);
            tmem_ld_wait(x);
            const uint32_t vis =
                visible(sees.x - key0 - 32 * q, sees.y - key0 - 32 * q, oks >> (2 * q));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float mx = ninf;
#pragma unroll
              for (int k = 16 * g; k < 16 * g + 16; ++k)
                if ((vis >> k) & 1u) mx = fmaxf(mx, __uint_as_float(x[k]));
              if (mx != ninf) {
                mx *= of_group(k_scale, q, g);
                top = fmaxf(top, mx);
                both = fmaxf(both, mx + of_group(ve, q, g));
              }
            }
          }
        }
        const bool grow =
            fmaxf(both - d, top + (kLagLog2 - kScoreLagLog2)) + b > kPLog2 + kLagLog2;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          float f_sum = 1.0f, f = 1.0f;
          if (grow) raise_refs(top, both, b, d, f_sum, f);
          l *= f_sum;
          if (opaque(j) > 0 && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
            live = warp_wait(bars + kPvDone + 16 * c + 8 * (buf ^ 1u),
                             (uint32_t)(((j - 1) >> 1) & 1),
                             abort);
            if (!live) break;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < kD / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(o_col + 16 * q, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(o_col + 16 * q, o);
            }
          }
        }
        // P of 32 keys lies in 16 columns of scores already read
        if (!masked) {
          float shift[kG];
          float2 sum[kG];
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            shift[g] = fmaxf(ve[g] - d, kVFloorLog2);
            sum[g] = make_float2(0.0f, 0.0f);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int g = (32 * q + 2 * k) / kN;
              const float sh = shift[g] + b;
              float2 e = fma2_rn(make_float2(__uint_as_float(a[q][2 * k]),
                                             __uint_as_float(a[q][2 * k + 1])),
                                 make_float2(k_scale[g], k_scale[g]), make_float2(sh, sh));
              e = make_float2(ex2(e.x), ex2(e.y));
              sum[g] = add2_rn(sum[g], e);
              pk[k] = pack_f16(e.x, e.y);
            }
            tmem_st16_issue(s_col + 16 * q, pk);
          }
#pragma unroll
          for (int g = 0; g < kG; ++g) l = fmaf(sum[g].x + sum[g].y, ex2(-shift[g]), l);
        } else {
          const int2 sees = lds_int2(base + L::kOffSees + 8 * r);
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t x[32], pk[16];
            tmem_ld32_issue(s_col + 32 * q, x);
            tmem_ld_wait(x);
            const uint32_t vis =
                visible(sees.x - key0 - 32 * q, sees.y - key0 - 32 * q, oks >> (2 * q));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float shift = fmaxf(of_group(ve, q, g) - d, kVFloorLog2);
              const float sc = of_group(k_scale, q, g), sh = shift + b;
              float sum = 0.0f;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int at = 16 * g + 2 * k;
                float e0 = ex2(fmaf(__uint_as_float(x[at]), sc, sh));
                float e1 = ex2(fmaf(__uint_as_float(x[at + 1]), sc, sh));
                if (((vis >> at) & 1u) == 0u) e0 = 0.0f;
                if (((vis >> at) & 2u) == 0u) e1 = 0.0f;
                sum += e0 + e1;
                pk[8 * g + k] = pack_f16(e0, e1);
              }
              if ((vis >> (16 * g)) & 0xFFFFu) l = fmaf(sum, ex2(-shift), l);
            }
            tmem_st16_issue(s_col + 16 * q, pk);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bars + kPFull + 16 * c + 8 * buf);
      }
      // the result
      if (live)
        live = warp_wait(bars + kPvDone + 16 * c + 8 * (uint32_t)((n_tiles - 1) & 1),
                         (uint32_t)(((n_tiles - 1) >> 1) & 1), abort);
      if (live) {
        tc_fence_after();
        const bool store = r < vw.rows;
        const bool whole = vw.chunks == 1;
        const bool wide =  // rows of 32-byte alignment
            (((uint32_t)(uintptr_t)p.out | (uint32_t)p.o_token | (uint32_t)p.o_head) & 31u) == 0u;
        int h = vw.h0 + r;
        const int qi = (int)((uint32_t)h / (uint32_t)p.group);
        h += (vw.head - qi) * p.group;
        const int64_t token = vw.span.first_row + vw.q0 + qi;
        const unsigned long long nans = *nan_mask;
        const float inv = l != 0.0f ? exp2f(d) / l : 0.0f;
        const float lse2 = l != 0.0f ? log2f(l) - b : ninf;
        uint8_t* to = p.out + token * p.o_token + h * p.o_head;
        float* part =
            p.tile_partials + ((int64_t)vw.part * (2 * kTileM) + r) * kPartPitch<kD>;
#pragma unroll 1
        for (int q = 0; q < kD / 16; ++q) {
          uint32_t o[16];
          __syncwarp();  // (rows that nothing is stored for come here early)
          tmem_ld16(o_col + 16 * q, o);
          if (!store) continue;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            o[k] = l != 0.0f ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
          if (nans) {
            uint32_t bad = 0;
            const int key_base = vw.t0 * kTileK;
#pragma unroll 1
            for (int b = 0; b < 64; ++b) {
              if (((nans >> b) & 1ull) == 0) continue;
              const int tile = b < 32 ? vw.u0 + b : vw.u1 - 1 - (b - 32);
              const int2 sees = lds_int2(base + L::kOffSees + 8 * r);
              bad |= nan_elements(p, vw.seq, vw.head, tile * kTileK, key_base + sees.y,
                                  key_base + sees.x, 16 * q);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if ((bad >> k) & 1u) o[k] = 0x7FC00000u;
          }
          if (whole) {
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              u[i] = narrow2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]), half);
            if (wide) {
              st_v8(to + 32 * q, u);
            } else {
              st_v4(to + 32 * q, make_uint4(u[0], u[1], u[2], u[3]));
              st_v4(to + 32 * q + 16, make_uint4(u[4], u[5], u[6], u[7]));
            }
          } else {
            const uint32_t(&lo)[8] = reinterpret_cast<const uint32_t(&)[8]>(o[0]);
            const uint32_t(&hi)[8] = reinterpret_cast<const uint32_t(&)[8]>(o[8]);
            st_v8(part + 16 * q, lo);
            st_v8(part + 16 * q + 8, hi);
          }
        }
        if (store) {
          if (!whole)
            part[kD] = lse2;
          else if (p.lse)
            p.lse[lse_place(token, p.heads, h)] = lse2 * 0.69314718055994531f;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort && p.status) atomicExch(p.status, 1);
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of every split unit: a warp takes a row, each lane kD / 32
// elements.
template <int kD>
__global__ void __launch_bounds__(256) fp8_attention_tiles_join_kernel(const Fp8AttnParams p) {
  constexpr int kE = kD / 32;
  const float ninf = neg_inf();
  const uint32_t y = blockIdx.x;
  int seq;
  uint32_t before;
  TileWork w = {};
  if (find_unit<256>(p, y, seq, before)) w = tile_work(p, seq, (int)(y - before), 0);
  // (on every path: a grid that ended before the one ahead of it would let the
  // next one start too early)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (w.chunks <= 1) return;  // no unit, or written whole
  const int head = blockIdx.y, lane = threadIdx.x & 31;
  for (int r = blockIdx.z * 8 + (threadIdx.x >> 5); r < w.rows; r += gridDim.z * 8) {
    const float* from =
        p.tile_partials +
        (((int64_t)y * p.kv_heads + head) * p.tile_chunks * (2 * kTileM) + r) * kPartPitch<kD>;
    const int64_t step = (int64_t)(2 * kTileM) * kPartPitch<kD>;
    // lane: one part's log-sum-exp (at most 16 parts)
    const float e = lane < w.chunks ? from[lane * step + kD] : ninf;
    float mx = e;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    mx = __shfl_sync(0xFFFFFFFFu, mx, 0);
    // root of the part's weight, 0 without keys
    const float weight = root_ex2(e - (mx == ninf ? 0.0f : mx));
    float sum = weight * weight, acc[kE];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    // (the mean at once: the sum of the parts may be too large)
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int k = 0; k < kE; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < w.chunks; ++c) {
      const float f = __shfl_sync(0xFFFFFFFFu, weight, c);
#pragma unroll
      for (int k = 0; k < kE; ++k)
        acc[k] = fmaf(from[c * step + kE * lane + k] * f, f * inv, acc[k]);
    }
    if (mx == ninf) mx = 0.0f;
    int qi, h;
    row_place(p, w, r, qi, h);
    h += head * p.group;
    uint8_t* to = p.out + (w.span.first_row + qi) * p.o_token + h * p.o_head + 2 * kE * lane;
#pragma unroll
    for (int k = 0; k < kE; k += 2)
      st_u32(to + 2 * k, narrow2(acc[k], acc[k + 1], p.half != 0));
    if (lane == 0 && p.lse)
      p.lse[lse_place(w.span.first_row + qi, p.heads, h)] =
          sum != 0.0f ? (mx + log2f(sum)) * 0.69314718055994531f : ninf;
  }
}

template <int kD, int kG>
int launch(const Fp8AttnParams& p, cudaStream_t stream) {
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
  if (!attr_done[dev]) {
    // (a build that launches with fewer registers than the roles share out
    // would wait for them without end)
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, fp8_attention_tiles_kernel<kD, kG>) != cudaSuccess ||
        attr.numRegs * kTileThreads < kBlockRegs ||
        cudaFuncSetAttribute(fp8_attention_tiles_kernel<kD, kG>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Layout<kD>::kBytes) != cudaSuccess) {
      cudaGetLastError();
      return KVQ_ECUDA;
    }
    attr_done[dev] = 1;
  }
  const int64_t grid = p.tile_units * p.kv_heads * p.tile_chunks;
  fp8_attention_tiles_kernel<kD, kG>
      <<<(unsigned)grid, kTileThreads, Layout<kD>::kBytes, stream>>>(p);
  const int rc = launch_status();
  if (rc != KVQ_OK || p.tile_chunks == 1) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tile_units, (unsigned)p.kv_heads, 16);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fp8_attention_tiles_join_kernel<kD>, p) != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  return launch_status();
}

}  // namespace

int64_t fp8_tiles_workspace(int64_t units, int64_t kv_heads, int chunks, int64_t head_dim) {
  return chunks > 1 ? units * kv_heads * chunks * 2 * kTileM * (head_dim + 8) * 4 : 0;
}

int fp8_tiles_launch(const Fp8AttnParams& p, int64_t head_dim, cudaStream_t stream) {
  const int log2 = p.cache.page_log2;
  if (head_dim == 128)
    return log2 >= 6 ? launch<128, 1>(p, stream)
                     : (log2 == 5 ? launch<128, 2>(p, stream) : launch<128, 4>(p, stream));
  return log2 >= 6 ? launch<64, 1>(p, stream)
                   : (log2 == 5 ? launch<64, 2>(p, stream) : launch<64, 4>(p, stream));
}

}  // namespace kvq
