// fp8_attention_tiles.cu — the tile kernel of fp8_paged_attention: many query
// rows of a key head (prompts, chunks of prompts, wide groups of heads) on
// the tcgen05 tensor cores, and the kernel that joins its partial results.
//
//   x_j = q . k_j * 2**ek(page) * sm_scale,  p_j = 2**(x_j - m),
//   out = sum_j p_j v_j * 2**ev(page) / sum_j p_j
//
// A block takes 256 query rows (queries x the heads of one key head) of a
// sequence as two tiles of 128, and the 128-key tiles that some row sees.
// E4M3 codes are exact in fp16, so both products run as kind::f16 with fp16
// operands and fp32 accumulators (M 128, N 128, K 16). Roles:
//   - producers (warps 8-11): codes from the pages into registers a tile
//     ahead, widened to fp16 into 128-byte-swizzled shared memory: keys are
//     read K-major, values MN-major from the same layout (two stages each).
//     They also work out each tile's page scales for the softmax;
//   - issuers (warps 12 and 13, one thread each, one for each row tile): S =
//     Q K^T, then O += P V and the next S, whose columns P occupies until
//     that product has completed. Two chains, so that one's softmax runs
//     while the tensor core works for the other;
//   - softmax (warps 0-3 and 4-7, a row per thread): reads S twice from
//     tensor memory (maximum, then probabilities), writes P as fp16 pairs
//     over it.
// The page scales are powers of two. A key's enters with the softmax scale; a
// value's is added to the exponent of the probability that enters the second
// product, relative to a reference that all rows share, and taken out again
// of the normaliser's sum.
//
// Few row tiles (a chunk behind a long context) are split over the keys as
// well, so that the grid fills the SMs; a second kernel joins the parts.
#include "fp8_attention.cuh"
#include "tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTileM = 128;  // rows of a tile
constexpr int kTileK = 128;  // keys of a tile
constexpr int kGroups = kTileK / 16;
constexpr int kTileThreads = 448;
constexpr int kProducerWarp = 8, kIssuerWarp = 12;
constexpr int kMetaSlots = 4;

// What the softmax needs of a tile's pages, by groups of 16 keys.
struct TileMeta {
  float k_scale[kGroups];  // 2**ek
  float shift[kGroups];    // ev - reference, at least kVFloorLog2
  float back[kGroups];     // 2**-shift
  float v_factor;          // what the sums of values take on before this tile
  float v_ref;
  uint32_t ok;             // groups whose page is in range
  uint32_t pad;
};

template <int kD>
struct Layout {
  static constexpr uint32_t kBlocks = kD / 64;                  // K-blocks of 64 elements
  static constexpr uint32_t kQBlock = 2 * kTileM * 128;         // 256 rows of 128 bytes
  static constexpr uint32_t kKvBlock = kTileK * 128;
  static constexpr uint32_t kStage = kBlocks * kKvBlock;
  static constexpr uint32_t kOffK = kBlocks * kQBlock;
  static constexpr uint32_t kOffV = kOffK + 2 * kStage;
  static constexpr uint32_t kOffMeta = kOffV + 2 * kStage;
  static constexpr uint32_t kOffQs = kOffMeta + kMetaSlots * sizeof(TileMeta);
  static constexpr uint32_t kOffBar = kOffQs + 2 * kTileM * 4;
  static constexpr uint32_t kOffEnd = kOffBar + 256;
  static constexpr size_t kBytes = kOffEnd + 1024;  // room to align the base
  static constexpr uint32_t kIdescQk = instr_desc(kTileM, kTileK, false, false);
  static constexpr uint32_t kIdescPv = instr_desc(kTileM, kD, true, false);
};

// mbarriers
constexpr uint32_t kKFull = 0, kVFull = 16, kKEmpty = 32, kVEmpty = 48;  // two stages each
constexpr uint32_t kSFull = 64, kPFull = 80, kPvDone = 96;               // one for each row tile
constexpr uint32_t kDrain = 112;                                         // one for each issuer
constexpr uint32_t kMeta = 128;                                          // kMetaSlots
constexpr uint32_t kTmemSlot = 176, kAbort = 184, kNanMask = 192;
static_assert(kMeta + 8 * kMetaSlots <= kTmemSlot, "mbarriers overlap");

__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
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

// Waits for this thread's tensor memory loads; the registers that they fill
// pass through, so that no use moves ahead of the wait.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
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

__device__ __forceinline__ bool nan_code(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
}
__device__ __forceinline__ uint32_t numbers_of(uint32_t w) {  // NaN codes cleared
  const uint32_t n = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return w & ~((n >> 7) * 0xFFu);
}

// Keeps the compiler from peeling a loop's first turns, or from copying the
// loop for each value of a condition (the kernel's code has to stay small: at twice the size, instruction fetches took most of the time).
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
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
};

__device__ __forceinline__ uint32_t tile_units(const Fp8AttnParams& p, int s) {
  const int rows = seq_span(p, s).n * p.group;
  return rows > p.row_limit ? (uint32_t)(rows + 2 * kTileM - 1) / (2 * kTileM) : 0u;
}

__device__ __forceinline__ TileWork tile_work(const Fp8AttnParams& p, int s, int unit, int chunk) {
  TileWork w;
  w.span = seq_span(p, s);
  w.row0 = unit * 2 * kTileM;
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
  w.t0 = min(w.u0 + chunk * per, w.u1);
  w.t1 = min(w.t0 + per, w.u1);
  return w;
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
// [d, d + 32): a rare path, straight from the cache.
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
    for (int i = 0; i < 32; ++i) bad |= (row[i] & 0x7F) == 0x7F ? 1u << i : 0u;
  }
  return bad;
}

// ---------------------------------------------------------------- producer ---

template <int kD>
struct Producer {
  static constexpr int kPieces = kD / 16;             // 16-byte pieces of a row
  static constexpr int kRowsAtOnce = 128 / kPieces;   // rows the 128 threads cover
  static constexpr int kLoads = kTileK / kRowsAtOnce;

  // Lane l < kGroups: where the codes of group l of a tile start (from the
  // caches' bases; -1: no page or no token), and the scales of its page.
  struct Pages {
    int64_t at;
    uint32_t ks, vs;
  };

  static __device__ __forceinline__ Pages pages(const Fp8AttnParams& p, const int64_t* table,
                                                int head, int tile, int end, int keys) {
    Pages r;
    r.at = -1;
    r.ks = r.vs = 127u;
    const int token = tile * kTileK + 16 * (threadIdx.x & 31);
    if ((threadIdx.x & 31) < kGroups && tile < end && token < keys) {
      const int64_t g = table[token >> p.cache.page_log2];
      if ((uint64_t)g < (uint64_t)p.cache.num_pages) {
        const int64_t sat = g * p.cache.scale_page_stride + head;
        r.ks = ld_u8(p.cache.k_scales + sat);
        r.vs = ld_u8(p.cache.v_scales + sat);
        r.at = g * p.cache.page_stride + head * p.cache.head_stride +
               (int64_t)(token & ((1 << p.cache.page_log2) - 1)) * p.cache.slot_stride;
      }
    }
    return r;
  }

  // A thread's pieces of a tile: rows i * kRowsAtOnce + its own (`off`: its
  // offset from the start of its row's group). `left`: tokens from the
  // thread's first row to the sequence's end; rows past it are zeros, like
  // those without a page.
  static __device__ __forceinline__ void load(const uint8_t* codes, const Pages& pg, int first_group,
                                              int64_t off, int left, uint4 (&out)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t at = __shfl_sync(0xFFFFFFFFu, pg.at, first_group + i * kRowsAtOnce / 16);
      out[i] = ld_codes(codes + at + off, at >= 0 && i * kRowsAtOnce < left);
    }
  }

  // 16 codes as fp16 into a stage: two 16-byte chunks of a swizzled row
  // (`at0`, `at1`: this thread's, for row 0 of each round; rounds are whole
  // groups of 8 rows apart, so the swizzle is the same). With 8 pieces to a
  // row the upper four store their chunks in the other order, so that the
  // eight lanes of a store phase cover all banks.
  static __device__ __forceinline__ void store(uint32_t at0, uint32_t at1, int i, bool swap,
                                               uint4 c) {
    uint32_t a0 = c.x, a1 = c.y, b0 = c.z, b1 = c.w;
    if (kPieces == 8 && swap) {
      a0 = c.z;
      a1 = c.w;
      b0 = c.x;
      b1 = c.y;
    }
    uint4 a, b;
    e4m3x4_to_f16x4(a0, a.x, a.y);
    e4m3x4_to_f16x4(a1, a.z, a.w);
    e4m3x4_to_f16x4(b0, b.x, b.y);
    e4m3x4_to_f16x4(b1, b.z, b.w);
    sts_v4(at0 + i * kRowsAtOnce * 128, a);
    sts_v4(at1 + i * kRowsAtOnce * 128, b);
  }
};

// ------------------------------------------------------------------ kernel ---

template <int kD>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp8_attention_tiles_kernel(const __grid_constant__ Fp8AttnParams p) {
  using L = Layout<kD>;
  using P = Producer<kD>;
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float ninf = neg_inf();

  // this block's unit: row tiles from the last to the first (under a causal
  // mask the longest first), and for each its key heads and parts
  const uint32_t wide = (uint32_t)p.kv_heads * (uint32_t)p.tile_chunks;
  const uint32_t y = blockIdx.x / wide;
  const uint32_t x = blockIdx.x - y * wide;
  const int head = (int)(x / (uint32_t)p.tile_chunks);
  const int chunk = (int)(x - (uint32_t)head * (uint32_t)p.tile_chunks);
  int seq;
  uint32_t before, total;
  const auto reversed = [&](int i) -> uint32_t { return tile_units(p, p.seqs.count - 1 - i); };
  if (!find_share<kTileThreads>(p.seqs.count, reversed, [&](uint32_t) { return y; }, seq, before,
                                total))
    return;
  seq = p.seqs.count - 1 - seq;
  const TileWork w = tile_work(p, seq, (int)(tile_units(p, seq) - 1 - (y - before)), chunk);
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
        if (c == 0 && p.lse) p.lse[(int64_t)(w.span.first_row + qi) * p.heads + h] = ninf;
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

  if (warp == kIssuerWarp) tmem_alloc(smem_addr(tmem_slot), 512);
  if (tid == 0) {
    const uint32_t chains = two ? 2 : 1;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + kKFull + 8 * i, 128);
      mbar_init(bars + kVFull + 8 * i, 128);
      mbar_init(bars + kKEmpty + 8 * i, chains);
      mbar_init(bars + kVEmpty + 8 * i, chains);
      mbar_init(bars + kSFull + 8 * i, 1);
      mbar_init(bars + kPFull + 8 * i, 128);
      mbar_init(bars + kPvDone + 8 * i, 1);
      mbar_init(bars + kDrain + 8 * i, 1);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(bars + kMeta + 8 * i, 1);
    *abort = 0;
    *nan_mask = 0ull;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // producers start their first loads while the softmax warps bring in Q
  const int pt = tid - 32 * kProducerWarp;
  const bool producer = pt >= 0 && pt < 128;
  const int prow = producer ? pt / P::kPieces : 0, piece = producer ? pt % P::kPieces : 0;
  const int64_t p_off = (int64_t)(prow & 15) * p.cache.slot_stride + 16 * piece;
  const int64_t* table = p.cache.table + seq * p.cache.table_stride;
  const int keys = w.span.keys;
  uint4 kb[P::kLoads], vb[P::kLoads];
  typename P::Pages pg = {-1, 127u, 127u}, pg_next = pg;
  if (producer) {
    pg = P::pages(p, table, head, w.t0, w.t1, keys);
    P::load(p.cache.k, pg, prow >> 4, p_off, keys - w.t0 * kTileK - prow, kb);
    P::load(p.cache.v, pg, prow >> 4, p_off, keys - w.t0 * kTileK - prow, vb);
    pg_next = P::pages(p, table, head, w.t0 + 1, w.t1, keys);
  } else if (tid < 256) {
    // rows as fp16, each times a power of two that brings its largest
    // magnitude to [2**14, 2**15); kD / 8 threads to a row
    constexpr int kT = kD / 8;
    const int c = tid % kT;
    constexpr int kAtOnce = 256 / kT, kBatch = 4;
#pragma unroll 1
    for (int r0 = tid / kT; r0 < 2 * kTileM; r0 += kAtOnce * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b * kAtOnce;
        v[b] = make_uint4(0, 0, 0, 0);
        if (r < w.rows) {
          int qi, h;
          row_place(p, w, r, qi, h);
          v[b] = ld_once_v4(p.q + (w.span.first_row + qi) * p.q_token +
                            (head * p.group + h) * p.q_head + 16 * c);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b * kAtOnce;
        float f[8];
        widen8(v[b], half, f);
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
#pragma unroll
        for (int o = 1; o < kT; o <<= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const int e = amax > 0.0f ? max((int)(__float_as_uint(amax) >> 23), 16) - 127 : 0;
        const float up = __uint_as_float((uint32_t)(min(14 - e, 127) + 127) << 23);
        if (c == 0) q_scale[r] = p.scale_log2 / up;
        const uint32_t at = base + (uint32_t)(c >> 3) * L::kQBlock + (uint32_t)r * 128 +
                            ((((uint32_t)c & 7) ^ ((uint32_t)r & 7)) << 4);
        sts_v4(at, make_uint4(pack_f16(f[0] * up, f[1] * up), pack_f16(f[2] * up, f[3] * up),
                              pack_f16(f[4] * up, f[5] * up), pack_f16(f[6] * up, f[7] * up)));
      }
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kColO = 256;

  if (producer) {
    // ------------------------------------------------------------ producers
    float v_ref = ninf;
    const uint32_t p_row = (uint32_t)(piece >> 2) * L::kKvBlock + (uint32_t)prow * 128;
    const uint32_t chunk0 = 2u * (uint32_t)(piece & 3), swz = (uint32_t)(prow & 7);
    const bool flip = P::kPieces == 8 && (piece & 4) != 0;
    const uint32_t p_at0 = base + L::kOffK + p_row + (((flip ? chunk0 + 1 : chunk0) ^ swz) << 4);
    const uint32_t p_at1 = base + L::kOffK + p_row + (((flip ? chunk0 : chunk0 + 1) ^ swz) << 4);
#pragma unroll 1
    for (int j = 0; j < n_tiles; ++j) {
      const int tile = w.t0 + j, key0 = tile * kTileK;
      const bool swap = opaque(flip) != 0;
      const uint32_t st = (uint32_t)(j & 1);
      const uint32_t parity = (uint32_t)(((j >> 1) - 1) & 1);  // 1 at first: passes at once
      const int left = j + 1 < n_tiles ? keys - key0 - kTileK - prow : 0;  // of the next tile
      if (!warp_wait(bars + kKEmpty + 8 * st, parity, abort)) break;
#pragma unroll
      for (int i = 0; i < P::kLoads; ++i)
        P::store(p_at0 + st * L::kStage, p_at1 + st * L::kStage, i, swap, kb[i]);
      fence_proxy_async();
      mbar_arrive(bars + kKFull + 8 * st);
      P::load(p.cache.k, pg_next, prow >> 4, p_off, left, kb);
      if (opaque(warp) == kProducerWarp) {
        // page scales of the tile's groups (lane = group)
        const bool ok = pg.at >= 0;
        const float ve = pg.vs == 255u ? 0.0f : e8m0_log2(pg.vs);
        float top = ok ? ve : ninf;
#pragma unroll
        for (int o = 1; o < kGroups; o <<= 1)
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        top = __shfl_sync(0xFFFFFFFFu, top, 0);
        float factor = 1.0f;
        if (top > v_ref + kVLagLog2) {
          factor = ex2(v_ref - top);
          v_ref = top;
        }
        const uint32_t oks = __ballot_sync(0xFFFFFFFFu, ok) & ((1u << kGroups) - 1u);
        TileMeta& m = meta[j & (kMetaSlots - 1)];
        if (lane < kGroups) {
          const float shift = ok ? fmaxf(ve - v_ref, kVFloorLog2) : 0.0f;
          m.k_scale[lane] = e8m0_value(pg.ks);
          m.shift[lane] = shift;
          m.back[lane] = ex2(-shift);
        }
        if (lane == 0) {
          m.v_factor = factor;
          m.v_ref = v_ref;
          m.ok = oks;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kMeta + 8 * (uint32_t)(j & (kMetaSlots - 1)));
      }

      if (!warp_wait(bars + kVEmpty + 8 * st, parity, abort)) break;
      // a tile that some row does not see whole: 0 * NaN is NaN, so a NaN that
      // not every row sees is kept out of the product, and the rows that see
      // it are told at the end; a page whose value scale is NaN holds NaN
      const bool partial = key0 + kTileK > w.all_lim || key0 < w.all_low;
      if (partial || __any_sync(0xFFFFFFFFu, pg.vs == 255u)) {
        bool found = false;
#pragma unroll
        for (int i = 0; i < P::kLoads; ++i) {
          const int r = i * P::kRowsAtOnce + prow;
          if (__shfl_sync(0xFFFFFFFFu, pg.vs, r >> 4) == 255u && key0 + r < keys)
            vb[i] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          if (partial) {
            found |= nan_code(vb[i].x) || nan_code(vb[i].y) || nan_code(vb[i].z) || nan_code(vb[i].w);
            vb[i] = make_uint4(numbers_of(vb[i].x), numbers_of(vb[i].y), numbers_of(vb[i].z),
                               numbers_of(vb[i].w));
          }
        }
        if (found) {
          // tiles at the lower edge from the unit's first, at the upper from
          // its last: a block's rows span at most 256 queries, so each has few
          const int from_low = tile - w.u0, from_high = w.u1 - 1 - tile;
          if (from_low < 32) atomicOr(nan_mask, 1ull << from_low);
          else if (from_high < 32) atomicOr(nan_mask, 1ull << (32 + from_high));
        }
      }
#pragma unroll
      for (int i = 0; i < P::kLoads; ++i)
        P::store(p_at0 + (2 + st) * L::kStage, p_at1 + (2 + st) * L::kStage, i, swap, vb[i]);
      fence_proxy_async();
      mbar_arrive(bars + kVFull + 8 * st);
      P::load(p.cache.v, pg_next, prow >> 4, p_off, left, vb);
      pg = pg_next;
      pg_next = P::pages(p, table, head, tile + 2, w.t1, keys);
    }
  } else if (warp >= kIssuerWarp) {
    // -------------------------------------------------------------- issuers
    const uint32_t c = (uint32_t)(warp - kIssuerWarp);  // row tile
    if (lane == 0 && (c == 0 || two)) {
      const uint64_t q_desc = smem_desc(base + c * (kTileM * 128), 16, 1024, 2);
      const uint64_t k_desc0 = smem_desc(base + L::kOffK, 16, 1024, 2);
      const uint64_t v_desc0 = smem_desc(base + L::kOffV, L::kKvBlock, 1024, 2);
      const uint32_t s_col = tmem + c * 128, o_col = tmem + kColO + c * kD;
      // Turn i: the product of values for tile i - 1 once P is there, then the
      // scores of tile i, which take the columns that P occupied.
#pragma unroll 1
      for (int i = 0; i <= n_tiles; ++i) {
        if (opaque(i) > 0) {
          const int j = i - 1;
          const uint32_t st = (uint32_t)(j & 1);
          if (!mbar_wait(bars + kVFull + 8 * st, (uint32_t)((j >> 1) & 1), abort) ||
              !mbar_wait(bars + kPFull + 8 * c, (uint32_t)(j & 1), abort))
            break;
          tc_fence_after();
          const uint64_t v_desc = desc_at(v_desc0, st * L::kStage);
#pragma unroll
          for (uint32_t ks = 0; ks < kTileK / 16; ++ks)
            mma_ts(o_col, s_col + 8 * ks, desc_at(v_desc, ks * 2048), L::kIdescPv,
                   j != 0 || ks != 0);
          mma_commit(bars + kPvDone + 8 * c);
          mma_commit(bars + kVEmpty + 8 * st);
        }
        if (i < n_tiles) {
          const uint32_t st = (uint32_t)(i & 1);
          if (!mbar_wait(bars + kKFull + 8 * st, (uint32_t)((i >> 1) & 1), abort) ||
              !mbar_wait(bars + kPvDone + 8 * c, (uint32_t)((i - 1) & 1), abort))
            break;
          tc_fence_after();
          const uint64_t k_desc = desc_at(k_desc0, st * L::kStage);
#pragma unroll
          for (uint32_t b = 0; b < L::kBlocks; ++b)
#pragma unroll
            for (uint32_t ks = 0; ks < 4; ++ks)
              mma_ss(s_col, desc_at(q_desc, b * L::kQBlock + ks * 32),
                     desc_at(k_desc, b * L::kKvBlock + ks * 32), L::kIdescQk, (b | ks) != 0);
          mma_commit(bars + kSFull + 8 * c);
          mma_commit(bars + kKEmpty + 8 * st);
        }
      }
      if (!drain_mmas(bars + kDrain + 8 * c)) *abort = 1;
    }
    __syncwarp();
  } else if (warp < 4 || two) {
    // -------------------------------------------------------------- softmax
    const uint32_t c = (uint32_t)(warp >> 2);
    const int r = tid;  // row of the block
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + c * 128, o_col = tmem + lanes + kColO + c * kD;
    const float qs = q_scale[r];
    // keys the row sees, from the block's first tile on
    const int key_base = w.t0 * kTileK;
    int lim = 0x7FFFFFFF, low = -0x7FFFFFFF, qi = 0, h = 0;
    if (r < w.rows) {
      row_place(p, w, r, qi, h);
      h += head * p.group;
      int lo, hi;
      key_range(p, w.span, qi, qi + 1, lo, hi);
      lim = hi - key_base;
      low = lo - key_base;
    }
    float m = ninf, l = 0.0f, v_ref = ninf;
    bool live = true;
#pragma unroll 1
    for (int j = 0; j < n_tiles; ++j) {
      const uint32_t slot = (uint32_t)(j & (kMetaSlots - 1));
      live = warp_wait(bars + kMeta + 8 * slot, (uint32_t)((j / kMetaSlots) & 1), abort) &&
             warp_wait(bars + kSFull + 8 * c, (uint32_t)(j & 1), abort);
      if (!live) break;
      tc_fence_after();
      const TileMeta& mt = meta[slot];
      const int key0 = j * kTileK;
      const uint32_t oks = mt.ok;
      const bool masked = __any_sync(0xFFFFFFFFu, key0 + kTileK > lim || key0 < low) ||
                          oks != (1u << kGroups) - 1u;
      // the row's visible keys of this tile: [vis_lo, vis_lo + vis_n)
      const int vis_lo = max(low - key0, 0);
      const uint32_t vis_n = (uint32_t)max(min(lim - key0, kTileK) - vis_lo, 0);
      float top = ninf;
      if (!masked) {
        uint32_t a[2][32];
        tmem_ld32_issue(s_col, a[0]);
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            tmem_ld_wait(a[u]);
            if (u == 0 || q == 0) tmem_ld32_issue(s_col + 32 * (q + u + 1), a[u ^ 1]);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float mx = __uint_as_float(a[u][16 * g]);
#pragma unroll
              for (int k = 1; k < 15; k += 2)
                mx = fmaxf(mx, fmaxf(__uint_as_float(a[u][16 * g + k]),
                                     __uint_as_float(a[u][16 * g + k + 1])));
              mx = fmaxf(mx, __uint_as_float(a[u][16 * g + 15]));
              top = fmaxf(top, mx * (qs * mt.k_scale[2 * (q + u) + g]));
            }
          }
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t a[32];
          tmem_ld32(s_col + 32 * q, a);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float mx = ninf;
            const int from = 32 * q + 16 * g - vis_lo;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if ((uint32_t)(from + k) < vis_n) mx = fmaxf(mx, __uint_as_float(a[16 * g + k]));
            if (mx != ninf && (oks >> (2 * q + g)) & 1u)
              top = fmaxf(top, mx * (qs * mt.k_scale[2 * q + g]));
          }
        }
      }
      const float factor = mt.v_factor;
      v_ref = mt.v_ref;
      const bool grow = top > m + kLagLog2;
      if (__any_sync(0xFFFFFFFFu, grow) || factor != 1.0f) {
        float f = 1.0f;
        if (grow) {
          f = ex2(m - top);
          m = top;
        }
        l *= f;
        f *= factor;
        if (opaque(j) > 0) {
          live = warp_wait(bars + kPvDone + 8 * c, (uint32_t)((j - 1) & 1), abort);
          if (!live) break;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < kD / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_col + 32 * q, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(o_col + 32 * q, o);
          }
        }
      }
      const float mu = kPLog2 - (m == ninf ? 0.0f : m);
      // P's columns 16 q .. 16 q + 15 lie in score columns already read
      if (!masked) {
        uint32_t a[2][32];
        tmem_ld32_issue(s_col, a[0]);
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            tmem_ld_wait(a[u]);
            if (u == 0 || q == 0) tmem_ld32_issue(s_col + 32 * (q + u + 1), a[u ^ 1]);
            uint32_t pk[16];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int gi = 2 * (q + u) + g;
              const float sc = qs * mt.k_scale[gi], sh = mt.shift[gi] + mu;
              const float2 sc2 = make_float2(sc, sc), sh2 = make_float2(sh, sh);
              float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                float2 e = fma2_rn(make_float2(__uint_as_float(a[u][16 * g + k]),
                                               __uint_as_float(a[u][16 * g + k + 1])),
                                   sc2, sh2);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                sum = add2_rn(sum, e);
                pk[8 * g + k / 2] = pack_f16(e.x, e.y);
              }
              l = fmaf(sum.x + sum.y, mt.back[gi], l);
            }
            tmem_st16_issue(s_col + 16 * (q + u), pk);
          }
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t a[32], pk[16];
          tmem_ld32(s_col + 32 * q, a);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int gi = 2 * q + g;
            const float sc = qs * mt.k_scale[gi], sh = mt.shift[gi] + mu;
            const int from = 16 * gi - vis_lo;
            const uint32_t n = (oks >> gi) & 1u ? vis_n : 0u;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float e0 = ex2(fmaf(__uint_as_float(a[16 * g + k]), sc, sh));
              float e1 = ex2(fmaf(__uint_as_float(a[16 * g + k + 1]), sc, sh));
              if ((uint32_t)(from + k) >= n) e0 = 0.0f;
              if ((uint32_t)(from + k + 1) >= n) e1 = 0.0f;
              sum += e0 + e1;
              pk[8 * g + k / 2] = pack_f16(e0, e1);
            }
            l = fmaf(sum, mt.back[gi], l);
          }
          tmem_st16_issue(s_col + 16 * q, pk);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bars + kPFull + 8 * c);
    }
    // the result
    if (live)
      live = warp_wait(bars + kPvDone + 8 * c, (uint32_t)((n_tiles - 1) & 1), abort);
    if (live) {
      tc_fence_after();
      const bool store = r < w.rows;
      const bool whole = w.chunks == 1;
      const unsigned long long nans = *nan_mask;
      const float inv = l != 0.0f ? exp2f(v_ref) / l : 0.0f;
      const float lse2 = l != 0.0f ? m + log2f(l) - kPLog2 : ninf;
      uint8_t* to = p.out + (w.span.first_row + qi) * p.o_token + h * p.o_head;
      float* part = p.tile_partials +
                    ((((int64_t)y * p.kv_heads + head) * p.tile_chunks + chunk) * (2 * kTileM) + r) *
                        (kD + 4);
#pragma unroll 1
      for (int q = 0; q < kD / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(o_col + 32 * q, o);
        if (!store) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = l != 0.0f ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
        if (nans) {
          uint32_t bad = 0;
#pragma unroll 1
          for (int b = 0; b < 64; ++b) {
            if (((nans >> b) & 1ull) == 0) continue;
            const int tile = b < 32 ? w.u0 + b : w.u1 - 1 - (b - 32);
            bad |= nan_elements(p, seq, head, tile * kTileK, key_base + low, key_base + lim, 32 * q);
          }
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if ((bad >> k) & 1u) o[k] = 0x7FC00000u;
        }
        if (whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              u[i] = narrow2(__uint_as_float(o[8 * k + 2 * i]), __uint_as_float(o[8 * k + 2 * i + 1]),
                             half);
            st_v4(to + 64 * q + 16 * k, make_uint4(u[0], u[1], u[2], u[3]));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_v4(part + 32 * q + 4 * k,
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
        }
      }
      if (store) {
        if (!whole)
          part[kD] = lse2;
        else if (p.lse)
          p.lse[(int64_t)(w.span.first_row + qi) * p.heads + h] = lse2 * 0.69314718055994531f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort && p.status) atomicExch(p.status, 1);
  if (warp == kIssuerWarp) {
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
  uint32_t before, total;
  const auto reversed = [&](int i) -> uint32_t { return tile_units(p, p.seqs.count - 1 - i); };
  if (!find_share<256>(p.seqs.count, reversed, [&](uint32_t) { return y; }, seq, before, total))
    return;
  seq = p.seqs.count - 1 - seq;
  const TileWork w = tile_work(p, seq, (int)(tile_units(p, seq) - 1 - (y - before)), 0);
  if (w.chunks <= 1) return;  // written whole
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int head = blockIdx.y, lane = threadIdx.x & 31;
  for (int r = blockIdx.z * 8 + (threadIdx.x >> 5); r < w.rows; r += gridDim.z * 8) {
    const float* from =
        p.tile_partials +
        (((int64_t)y * p.kv_heads + head) * p.tile_chunks * (2 * kTileM) + r) * (kD + 4);
    const int64_t step = (int64_t)(2 * kTileM) * (kD + 4);
    float mx = ninf;
    for (int c = 0; c < w.chunks; ++c) mx = fmaxf(mx, from[c * step + kD]);
    if (mx == ninf) mx = 0.0f;
    float sum = 0.0f, acc[kE];
#pragma unroll
    for (int k = 0; k < kE; ++k) acc[k] = 0.0f;
    for (int c = 0; c < w.chunks; ++c) {
      const float f = ex2(from[c * step + kD] - mx);  // 0 for a part without keys
      sum += f;
#pragma unroll
      for (int k = 0; k < kE; ++k) acc[k] = fmaf(from[c * step + kE * lane + k], f, acc[k]);
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    int qi, h;
    row_place(p, w, r, qi, h);
    h += head * p.group;
    uint8_t* to = p.out + (w.span.first_row + qi) * p.o_token + h * p.o_head + 2 * kE * lane;
#pragma unroll
    for (int k = 0; k < kE; k += 2)
      st_u32(to + 2 * k, narrow2(acc[k] * inv, acc[k + 1] * inv, p.half != 0));
    if (lane == 0 && p.lse)
      p.lse[(int64_t)(w.span.first_row + qi) * p.heads + h] =
          sum != 0.0f ? (mx + log2f(sum)) * 0.69314718055994531f : ninf;
  }
}

template <int kD>
int launch(const Fp8AttnParams& p, cudaStream_t stream) {
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ECUDA;
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(fp8_attention_tiles_kernel<kD>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Layout<kD>::kBytes) != cudaSuccess) {
      cudaGetLastError();
      return KVQ_ECUDA;
    }
    attr_done[dev] = 1;
  }
  const int64_t grid = p.tile_units * p.kv_heads * p.tile_chunks;
  fp8_attention_tiles_kernel<kD><<<(unsigned)grid, kTileThreads, Layout<kD>::kBytes, stream>>>(p);
  const int rc = launch_status();
  if (rc != KVQ_OK || p.tile_chunks == 1) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tile_units, (unsigned)p.kv_heads, 4);
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
  return chunks > 1 ? units * kv_heads * chunks * 2 * kTileM * (head_dim + 4) * 4 : 0;
}

int fp8_tiles_launch(const Fp8AttnParams& p, int64_t head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace kvq
