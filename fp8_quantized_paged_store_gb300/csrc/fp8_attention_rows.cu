// fp8_attention_rows.cu — the row kernel of fp8_paged_attention: few query
// rows of a key head (a decode step, a short run of drafted tokens) against a
// long cache, and the kernel that joins its partial results.
//
//   x_j = q . k_j * 2**ek(page) * sm_scale,  p_j = 2**(x_j - m),
//   out = sum_j p_j v_j * 2**ev(page) / sum_j p_j
//
// Bound by memory: the cache is read once, 2 * head_dim bytes a token and key
// head, while a row costs 4 * head_dim operations a token.
//
// Keys are the rows (M) of the first product and value elements the rows of
// the second, with the query rows as the 8 columns (N) of mma.m16n8k16, so
// every code is widened, E4M3 to fp16 exactly, by the one thread whose
// fragment it belongs to, two per instruction. The order of the summed
// dimension is free, so a thread's 16 consecutive key elements serve as its
// fragments; values are paired over two tokens by one byte permute. Scores
// turn from the first product's result layout into the second's operand
// layout by movmatrix.
//
// A warp takes tiles of 32 keys on its own (its own running maximum, sums and
// output) and loads them into a ring of its own in shared memory, kStages
// tiles ahead, by 16-byte asynchronous copies: no barrier in the loop, and
// some 150 KB in flight on an SM. All (sequence, key head) units' tiles are
// shared out evenly over one resident grid, whatever the lengths: a block's
// warps join their results of a unit in shared memory, and units that span
// blocks are joined by a second kernel from at most two partials a block.
//
// 64 single tokens against 500 to 16,000 keys in 8 key heads of 128: 171 us
// with the join, 6470 GB/s (95 % of a copy's rate); 16 rows (two tokens of
// eight heads) against 60,000 to 131,000 keys 145 us (92 %). The scores' scaling
// and the probabilities' exponents are packed pairs: one by one they took 176
// and 158 us. A call costs 5 us with a tile for each warp: two kernels' chains.
#include "fp8_attention.cuh"

namespace kvq {
namespace {

constexpr int kStages = 3;

// 16-byte asynchronous copy of codes, or 16 zero bytes.
__device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t* src, bool have) {
  const uint32_t n = have ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
// Issued where it stands: the tile that it belongs to comes kStages later.
__device__ __forceinline__ uint32_t ld_byte(const uint8_t* p) {
  uint32_t r;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A byte of w whose low seven bits are all ones (the E4M3 NaN)?
__device__ __forceinline__ bool has_nan_code(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
}
// 0xFF in every byte that is not the E4M3 NaN.
__device__ __forceinline__ uint32_t number_codes(uint32_t w) {
  const uint32_t n = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return ~((n >> 7) * 0xFFu);
}

// kD: head dim, kN: 8-row columns (rows <= 8 * kN), kSmallPage: pages of 16
// tokens, two to a tile.
template <int kD, int kN, bool kSmallPage>
struct RowKernel {
  static constexpr int kH = kD / 64;   // 16-byte pieces of a key row a thread takes
  static constexpr int kI = kD / 16;   // 16-row blocks of the output
  static constexpr int kRows = 8 * kN;
  static constexpr int kPages = kSmallPage ? 2 : 1;   // of a tile
  static constexpr uint32_t kTileBytes = kRowTokens * kD;  // keys or values
  static constexpr uint32_t kRing = kStages * 2 * kTileBytes;  // of a warp
  // after the loop the rings hold the warps' results
  static constexpr int kPitch = kD + 4;
  static constexpr uint32_t kJoin = kRowWarps * kRows * kPitch * 4;
  static constexpr uint32_t kBytes =
      kRowWarps * kRing > kJoin ? kRowWarps * kRing : kJoin;

  struct Pages {
    int64_t g[kPages];  // -1: none
  };
  struct Scales {
    uint32_t k[kPages], v[kPages];
    uint32_t ok;  // bit i: page i is in range
  };

  // `table`: the sequence's row of the block table.
  static __device__ __forceinline__ Pages pages(const Fp8AttnParams& p, const int64_t* table,
                                                int tile, int end, int keys) {
    Pages r;
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      const int token = tile * kRowTokens + 16 * i;
      r.g[i] = tile < end && token < keys ? table[token >> p.cache.page_log2] : -1;
    }
    return r;
  }

  // The page scales of a tile whose pages have been copied.
  static __device__ __forceinline__ Scales scales(const Fp8AttnParams& p, const Pages& pg,
                                                  int head) {
    Scales sc;
    sc.ok = 0;
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      const int64_t g = pg.g[i];
      const bool ok = (uint64_t)g < (uint64_t)p.cache.num_pages;
      const int64_t at = ok ? g * p.cache.scale_page_stride + head : 0;
      sc.k[i] = ok ? ld_byte(p.cache.k_scales + at) : 127u;
      sc.v[i] = ok ? ld_byte(p.cache.v_scales + at) : 127u;
      if (ok) sc.ok |= 1u << i;
    }
    return sc;
  }

  // Where piece `piece` of row `row` of a tile lies: conflict-free for the
  // fragment reads below. A key read takes two neighbouring rows' pieces t or
  // t + 4 at once; a value read rows 2t of one parity, pieces g and g + 1.
  static __device__ __forceinline__ uint32_t k_place(int row, int piece) {
    return (uint32_t)(row * kD + ((kD == 128 ? piece ^ ((row & 1) << 2) : piece) << 4));
  }
  static __device__ __forceinline__ uint32_t v_place(int row, int piece) {
    return (uint32_t)(row * kD + ((kD == 128 ? piece ^ (row & 6) : piece ^ (row & 2)) << 4));
  }

  // Copies a tile into a stage; rows without a page are zeros. Past the end an
  // empty group of copies.
  static __device__ __forceinline__ void copy(const Fp8AttnParams& p, const Pages& pg, int tile,
                                              int end, int head, uint32_t stage) {
    if (tile < end) fill(p, pg, tile, head, stage);
    cp_async_commit();
  }
  static __device__ __forceinline__ void fill(const Fp8AttnParams& p, const Pages& pg, int tile,
                                              int head, uint32_t stage) {
    constexpr int kPieces = kD / 16, kAtOnce = 32 / kPieces;
    constexpr int kCount = kRowTokens / kPages / kAtOnce;
    const int lane = threadIdx.x & 31;
    const int row0 = lane / kPieces, piece = lane % kPieces;
    const int64_t step = (int64_t)kAtOnce * p.cache.slot_stride;
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      const int64_t g = pg.g[i];
      const bool ok = (uint64_t)g < (uint64_t)p.cache.num_pages;
      const int slot = kSmallPage ? 0 : (tile * kRowTokens) & ((1 << p.cache.page_log2) - 1);
      const int64_t at = ok ? g * p.cache.page_stride + head * p.cache.head_stride +
                                  (int64_t)(slot + row0) * p.cache.slot_stride + 16 * piece
                            : 0;
      const uint8_t* k = p.cache.k + at;
      const uint8_t* v = p.cache.v + at;
#pragma unroll
      for (int c = 0; c < kCount; ++c) {
        const int row = i * (kRowTokens / kPages) + c * kAtOnce + row0;
        copy_codes(stage + k_place(row, piece), k, ok);
        if (ok) k += step;
      }
#pragma unroll
      for (int c = 0; c < kCount; ++c) {
        const int row = i * (kRowTokens / kPages) + c * kAtOnce + row0;
        copy_codes(stage + kTileBytes + v_place(row, piece), v, ok);
        if (ok) v += step;
      }
    }
  }
};

template <int kD, int kN, bool kSmallPage>
__global__ void __launch_bounds__(kRowThreads) fp8_attention_rows_kernel(
    const __grid_constant__ Fp8AttnParams p) {
  using K = RowKernel<kD, kN, kSmallPage>;
  constexpr int kH = K::kH, kI = K::kI, kRows = K::kRows;
  constexpr int kLast = K::kPages - 1;  // page of half h of a tile: kLast * h
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_b[kRowWarps][kRows], sm_d[kRowWarps][kRows], sm_l[kRowWarps][kRows];
  float* sm_o = reinterpret_cast<float*>(smem);  // [kRowWarps][kRows][kPitch]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const float ninf = neg_inf();
  const bool half = p.half != 0;

  // this block's share [at, end) of all tiles
  int seq;
  uint32_t before, total, at, end;
  const auto weight = [&](int s) -> uint32_t {
    const RowShare r = row_share(p, s);
    return r.tiles * r.units;
  };
  const auto place = [&](uint32_t sum) -> uint32_t {
    const uint32_t blocks = row_blocks(p, sum);
    if (blockIdx.x >= blocks) return sum;
    at = share_start(blockIdx.x, sum, blocks);
    end = share_start(blockIdx.x + 1, sum, blocks);
    return at;
  };
  if (!find_share<kRowThreads>(p.seqs.count, weight, place, seq, before, total)) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * K::kRing;
  RowShare sh = row_share(p, seq);
  while (at < end) {
    // the unit that holds tile `at`
    while (at >= before + sh.tiles * sh.units) {
      before += sh.tiles * sh.units;
      sh = row_share(p, ++seq);
    }
    const int unit = (int)((at - before) / sh.tiles);
    const uint32_t unit_start = before + unit * sh.tiles;
    // key head and rows [row0, row0 + rows) of the sequence
    const int head = sh.rows > kRows ? unit >> 1 : unit;
    const int row0 = sh.rows > kRows ? (unit & 1) * kRows : 0;
    const int rows = min(sh.rows - row0, kRows);
    const uint32_t seg_end = min(end, unit_start + sh.tiles);
    const int tile0 = sh.first + (int)(at - unit_start);
    const int tile1 = sh.first + (int)(seg_end - unit_start);
    const int64_t* table = p.cache.table + seq * p.cache.table_stride;

    // the first tiles on their way
    typename K::Pages pg[kStages];  // of this tile and the next ones
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      pg[i] = K::pages(p, table, tile0 + warp + i * kRowWarps, tile1, sh.span.keys);
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      K::copy(p, pg[i], tile0 + warp + i * kRowWarps, tile1, head, ring + i * 2 * K::kTileBytes);
    typename K::Scales sc_next = K::scales(p, pg[0], head);
    typename K::Pages pg_next =
        K::pages(p, table, tile0 + warp + kStages * kRowWarps, tile1, sh.span.keys);

    // query fragments: row 8 c + g, as fp16 times a power of two that brings
    // the row's largest magnitude to [2**14, 2**15)
    uint32_t qf[kN][kH][4][2];
    float qs[kN][2];                 // per result column: scale_log2 / that power
    int32_t lim[kN][2], low[kN][2];  // keys the column's row sees, from the segment's first
    const int base_key = tile0 * kRowTokens;
    int32_t all_lim = 0x7FFFFFFF, all_low = -0x7FFFFFFF;
    uint4 w[kN][kH][2];
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const int r = 8 * c + g;
      const bool have = r < rows;
      const int of_seq = row0 + (have ? r : 0);
      const int qi = (int)((uint32_t)of_seq / (uint32_t)p.group);
      const uint8_t* qrow = p.q + (sh.span.first_row + qi) * p.q_token +
                            (head * p.group + of_seq - qi * p.group) * p.q_head;
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[c][i][j] = have ? ld_nc_v4(qrow + 2 * (64 * i + 16 * t + 8 * j)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      // (by the bits of the 16-bit values)
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 x = w[c][i][j];
          top = max_u16x2(top, max_u16x2(max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                         max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
        }
      top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const float amax = widen2(max(top & 0xFFFFu, top >> 16), half).x;
      // amax in [2**e, 2**(e + 1)); scaled by 2**(14 - e)
      const int e = amax > 0.0f ? max((int)(__float_as_uint(amax) >> 23), 16) - 127 : 0;
      const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
      const float down = p.scale_log2 * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[8];
          widen8(w[c][i][j], half, f);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            qf[c][i][2 * j + k][0] = pack_f16x2(f[4 * k] * up, f[4 * k + 1] * up);
            qf[c][i][2 * j + k][1] = pack_f16x2(f[4 * k + 2] * up, f[4 * k + 3] * up);
          }
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // result column 2 t + j: its scale sits in lane group g' = 2 t + j
        qs[c][j] = __shfl_sync(0xFFFFFFFFu, down, 4 * (2 * t + j));
        const int col = 8 * c + 2 * t + j;
        const int qi = (int)((uint32_t)(row0 + (col < rows ? col : 0)) / (uint32_t)p.group);
        int lo, hi;
        key_range(p, sh.span, qi, qi + 1, lo, hi);
        lim[c][j] = hi - base_key;
        low[c][j] = lo - base_key;
        all_lim = min(all_lim, lim[c][j]);
        all_low = max(all_low, low[c][j]);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      all_lim = min(all_lim, __shfl_xor_sync(0xFFFFFFFFu, all_lim, o));
      all_low = max(all_low, __shfl_xor_sync(0xFFFFFFFFu, all_low, o));
    }

    float b[kN][2], d[kN][2], l[kN][2], o[kI][kN][4];
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      b[c][0] = b[c][1] = kNoKey;
      d[c][0] = d[c][1] = 0.0f;
      l[c][0] = l[c][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kI; ++i) o[i][c][0] = o[i][c][1] = o[i][c][2] = o[i][c][3] = 0.0f;
    }

    const int n_tiles = tile1 - tile0;
    uint32_t stage = 0;
#pragma unroll 1
    for (int it = warp; it < n_tiles; it += kRowWarps) {
      const uint32_t k_at = ring + stage * 2 * K::kTileBytes, v_at = k_at + K::kTileBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const typename K::Scales sc = sc_next;
      sc_next = K::scales(p, pg[1], head);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      // scores: two halves of 16 keys x 8 kN rows
      float s[2][kN][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < kN; ++c) s[h][c][0] = s[h][c][1] = s[h][c][2] = s[h][c][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kH; ++i) {
          const uint4 ka = lds16(k_at + K::k_place(16 * h + g, t + 4 * i));
          const uint4 kb = lds16(k_at + K::k_place(16 * h + g, t + 4 * i) + 8 * kD);
          const uint32_t a[4] = {ka.x, ka.y, ka.z, ka.w};
          const uint32_t bw[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w4 = 0; w4 < 4; ++w4) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(a[w4], a0, a2);
            e4m3x4_to_f16x4(bw[w4], a1, a3);
#pragma unroll
            for (int c = 0; c < kN; ++c)
              mma_f16(s[h][c], a0, a1, a2, a3, qf[c][i][w4][0], qf[c][i][w4][1]);
          }
        }
      }
      // page scales
      float ks[K::kPages], ve[K::kPages];
      bool ok[K::kPages], vnan[K::kPages];
#pragma unroll
      for (int i = 0; i < K::kPages; ++i) {
        ok[i] = (sc.ok >> i) & 1u;
        ks[i] = e8m0_value(sc.k[i]);
        vnan[i] = sc.v[i] == 255u;  // the page's values are NaN
        ve[i] = vnan[i] ? 0.0f : e8m0_log2(sc.v[i]);
      }
      // scaled scores; -inf where a row does not see the key
      const int32_t key0 = it * kRowTokens;
      const bool whole =
          ok[0] && ok[kLast] && key0 + kRowTokens <= all_lim && key0 >= all_low;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          const float k = ks[kLast * h];
          const float2 qk = mul2_rn(make_float2(qs[c][0], qs[c][1]), make_float2(k, k));
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 x = mul2_rn(make_float2(s[h][c][2 * r], s[h][c][2 * r + 1]), qk);
            s[h][c][2 * r] = x.x;
            s[h][c][2 * r + 1] = x.y;
          }
        }
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int32_t key = key0 + 16 * h + 8 * r + g;
#pragma unroll
            for (int c = 0; c < kN; ++c)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (!ok[kLast * h] || key >= lim[c][j] || key < low[c][j]) s[h][c][2 * r + j] = ninf;
          }
      }
      // a row's products are stored with the exponent of the values less d, and
      // both references taken out (see raise_refs)
      float dv[K::kPages][kN][2], shift[K::kPages][kN][2];
      const auto shifts = [&]() {
#pragma unroll
        for (int i = 0; i < K::kPages; ++i)
#pragma unroll
          for (int c = 0; c < kN; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              dv[i][c][j] = fmaxf(ve[i] - d[c][j], kVFloorLog2);
              shift[i][c][j] = dv[i][c][j] + b[c][j];
            }
      };
      shifts();
      bool grow = false;
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) top[h] = fmaxf(s[h][c][j], s[h][c][2 + j]);
          if (!kSmallPage) top[0] = fmaxf(top[0], top[1]);
#pragma unroll
          for (int i = 0; i < K::kPages; ++i)
            grow |= top[i] + fmaxf(dv[i][c][j], kLagLog2 - kScoreLagLog2) + b[c][j] >
                    kPLog2 + kLagLog2;
        }
      // rescale the sums when a row has outgrown its references
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (int c = 0; c < kN; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // the row's maxima over the tile: over the eight lanes that
            // hold its keys
            float tm = ninf, tb = ninf;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = fmaxf(s[h][c][j], s[h][c][2 + j]);
              tm = fmaxf(tm, x);
              tb = fmaxf(tb, x + ve[kLast * h]);
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              tm = fmaxf(tm, __shfl_xor_sync(0xFFFFFFFFu, tm, x));
              tb = fmaxf(tb, __shfl_xor_sync(0xFFFFFFFFu, tb, x));
            }
            float f_sum = 1.0f, f = 1.0f;
            if (fmaxf(tb - d[c][j], tm) + b[c][j] > kPLog2)
              raise_refs(tm, tb, b[c][j], d[c][j], f_sum, f);
            l[c][j] *= f_sum;
#pragma unroll
            for (int i = 0; i < kI; ++i) {
              o[i][c][j] *= f;
              o[i][c][2 + j] *= f;
            }
          }
        shifts();
      }
      // probabilities times 2**(kPLog2 + value exponent - d)
      uint32_t pf[2][kN][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          float pr[4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 x = add2_rn(make_float2(s[h][c][2 * r], s[h][c][2 * r + 1]),
                                     make_float2(shift[kLast * h][c][0], shift[kLast * h][c][1]));
            pr[2 * r] = ex2(x.x);
            pr[2 * r + 1] = ex2(x.y);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            l[c][j] = fmaf(pr[j] + pr[2 + j], ex2(-dv[kLast * h][c][j]), l[c][j]);
          // results are keys x rows, (row g, columns 2t, 2t + 1); the second
          // product wants (rows 2t, 2t + 1, column g)
          pf[h][c][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
          pf[h][c][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
        }
      }
      // output += V^T P^T: block i holds elements (kD / 8) g + 2 i (+ 1)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[4][kI / 2];  // token, words
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * h + 2 * t + (r & 1) + 8 * (r >> 1);
          if constexpr (kD == 128) {
            const uint4 x = lds16(v_at + K::v_place(row, g));
            v[r][0] = x.x;
            v[r][1] = x.y;
            v[r][2] = x.z;
            v[r][3] = x.w;
          } else {
            const uint2 x = lds8(v_at + K::v_place(row, g >> 1) + 8 * (g & 1));
            v[r][0] = x.x;
            v[r][1] = x.y;
          }
        }
        if (!whole || vnan[kLast * h]) {
          // values of keys that no row sees must not reach the product, where
          // 0 * NaN is NaN; a NaN that only some rows see is added to them
          const int32_t end_key = sh.span.keys - base_key;
          bool found = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int32_t key = key0 + 16 * h + 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
            for (int i = 0; i < kI / 2; ++i) {
              if (vnan[kLast * h]) v[r][i] = 0x7F7F7F7Fu;
              if (key >= end_key) v[r][i] = 0;
              found |= has_nan_code(v[r][i]);
            }
          }
          if (__any_sync(0xFFFFFFFFu, found)) {
            // a rare path: for every token, the quad's owner says which of
            // its elements are NaN, and the quad marks the rows that see it;
            // then the codes are cleared
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              const int owner = (k & 7) >> 1, r = (k & 1) + 2 * (k >> 3);
              uint32_t bad = 0;
#pragma unroll
              for (int rr = 0; rr < 4; ++rr)
                if (rr == r && owner == t) {
#pragma unroll
                  for (int i = 0; i < kI / 2; ++i) {
                    const uint32_t num = number_codes(v[rr][i]);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                      if (((num >> (8 * b)) & 1u) == 0u) bad |= 1u << (4 * i + b);
                  }
                }
              bad = __shfl_sync(0xFFFFFFFFu, bad, (lane & ~3) | owner);
              const int32_t key = key0 + 16 * h + k;
#pragma unroll
              for (int c = 0; c < kN; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (key < lim[c][j] && key >= low[c][j]) {
#pragma unroll
                    for (int i = 0; i < kI; ++i) {
                      if ((bad >> (2 * i)) & 1u) o[i][c][j] = __int_as_float(0x7FC00000);
                      if ((bad >> (2 * i + 1)) & 1u) o[i][c][2 + j] = __int_as_float(0x7FC00000);
                    }
                  }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int i = 0; i < kI / 2; ++i) v[r][i] &= number_codes(v[r][i]);
          }
        }
#pragma unroll
        for (int w4 = 0; w4 < kI / 2; ++w4) {
          const uint32_t x = prmt(v[0][w4], v[1][w4], 0x5140);
          const uint32_t y = prmt(v[2][w4], v[3][w4], 0x5140);
          const uint32_t x2 = prmt(v[0][w4], v[1][w4], 0x7362);
          const uint32_t y2 = prmt(v[2][w4], v[3][w4], 0x7362);
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          e4m3x4_to_f16x4(x, a0, a1);
          e4m3x4_to_f16x4(y, a2, a3);
          e4m3x4_to_f16x4(x2, b0, b1);
          e4m3x4_to_f16x4(y2, b2, b3);
#pragma unroll
          for (int c = 0; c < kN; ++c) {
            mma_f16(o[2 * w4][c], a0, a1, a2, a3, pf[h][c][0], pf[h][c][1]);
            mma_f16(o[2 * w4 + 1][c], b0, b1, b2, b3, pf[h][c][0], pf[h][c][1]);
          }
        }
      }
      // the stage's next tile
      __syncwarp();
      const int next = tile0 + it + kStages * kRowWarps;
      K::copy(p, pg_next, next, tile1, head, k_at);
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) pg[i] = pg[i + 1];
      pg[kStages - 1] = pg_next;
      pg_next = K::pages(p, table, next + kRowWarps, tile1, sh.span.keys);
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp's ring is free

    // join the block's warps
#pragma unroll
    for (int c = 0; c < kN; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[c][j] += __shfl_xor_sync(0xFFFFFFFFu, l[c][j], x);
        const int col = 8 * c + 2 * t + j;
        if (g == 0) {
          sm_b[warp][col] = b[c][j];
          sm_d[warp][col] = d[c][j];
          sm_l[warp][col] = l[c][j];
        }
        float* to = sm_o + (warp * kRows + col) * K::kPitch + (kD / 8) * g;
#pragma unroll
        for (int i = 0; i < kI; i += 2)
          *reinterpret_cast<float4*>(to + 2 * i) =
              make_float4(o[i][c][j], o[i][c][2 + j], o[i + 1][c][j], o[i + 1][c][2 + j]);
      }
    __syncthreads();
    const bool complete = at == unit_start && seg_end == unit_start + sh.tiles;
    const int64_t part = ((int64_t)blockIdx.x * 2 + (at == unit_start ? 1 : 0)) * kRows;
    // thread: 4 elements of a row
    for (int id = threadIdx.x; id < rows * (kD / 4); id += kRowThreads) {
      const int r = id / (kD / 4), e = 4 * (id - r * (kD / 4));
      // the warps' largest references (of warps without a key: far below)
      float mx = ninf, mo = ninf;
#pragma unroll
      for (int w4 = 0; w4 < kRowWarps; ++w4) {
        mx = fmaxf(mx, -sm_b[w4][r]);
        mo = fmaxf(mo, sm_d[w4][r] - sm_b[w4][r]);
      }
      // a row without keys has sum 0; one whose scores are all NaN has
      // none either and a NaN sum, which stays
      float sum = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w4 = 0; w4 < kRowWarps; ++w4) {
        const float f = ex2(-sm_b[w4][r] - mx);
        sum = fmaf(sm_l[w4][r], f, sum);
        const float fv = ex2(sm_d[w4][r] - sm_b[w4][r] - mo);
        const float4 x =
            *reinterpret_cast<const float4*>(sm_o + (w4 * kRows + r) * K::kPitch + e);
        acc.x = fmaf(x.x, fv, acc.x);
        acc.y = fmaf(x.y, fv, acc.y);
        acc.z = fmaf(x.z, fv, acc.z);
        acc.w = fmaf(x.w, fv, acc.w);
      }
      // (both factors at once: the sums may be too large for the first alone)
      const float inv = sum != 0.0f ? exp2f(mo - mx) / sum : 0.0f;
      const float lse2 = sum != 0.0f ? mx + log2f(sum) : ninf;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (complete) {
        const int qi = (int)((uint32_t)(row0 + r) / (uint32_t)p.group);
        const int h = head * p.group + row0 + r - qi * p.group;
        uint8_t* to = p.out + (sh.span.first_row + qi) * p.o_token + (int64_t)h * p.o_head + 2 * e;
        st_v2(to, narrow2(acc.x, acc.y, half), narrow2(acc.z, acc.w, half));
        if (e == 0 && p.lse)
          p.lse[lse_place(sh.span.first_row + qi, p.heads, h)] = lse2 * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4*>(p.row_partials + (part + r) * kD + e) = acc;
        if (e == 0) p.row_lse[part + r] = lse2;
      }
    }
    __syncthreads();
    at = seg_end;
  }
  // behind the tile kernel it may start early, but not end before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the partials of every unit that spans blocks: block (b, y) takes rows
// 4 y to 4 y + 3 (a warp each) of the unit that goes on from block b - 1 into
// block b, if it began there. The unit has a partial in each block that holds
// tiles of it. Blocks past those write zeros for sequences without a key. (A
// block for each sequence, head and row, most of them with nothing to join,
// took 4.3 ms for 4096 sequences of 200 keys, all together 0.5 ms so.)
template <int kD>
__global__ void __launch_bounds__(kRowThreads) fp8_attention_rows_join_kernel(
    const __grid_constant__ Fp8AttnParams p) {
  constexpr int kE = kD / 32;  // elements of a lane
  const float ninf = neg_inf();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = kRowWarps * (int)blockIdx.y + warp;  // of the unit
  if ((int)blockIdx.x >= p.row_grid) {
    const int s = ((int)blockIdx.x - p.row_grid) * kRowThreads + (int)threadIdx.x;
    RowShare sh = {};
    if (blockIdx.y == 0 && s < p.seqs.count) sh = row_share(p, s);
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, sh.rows > 0 && sh.tiles == 0);
    while (todo) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      const int first = __shfl_sync(0xFFFFFFFFu, sh.span.first_row, from);
      const int n = __shfl_sync(0xFFFFFFFFu, sh.span.n, from) * p.heads;
      constexpr int kPieces = kD / 8;  // of 16 bytes, in a row
      for (int i = lane / kPieces; i < n; i += 32 / kPieces) {
        const int64_t token = first + i / p.heads;
        const int h = i % p.heads, c = lane % kPieces;
        st_v4(p.out + token * p.o_token + h * p.o_head + 16 * c, make_uint4(0, 0, 0, 0));
        if (c == 0 && p.lse) p.lse[lse_place(token, p.heads, h)] = ninf;
      }
    }
    return;
  }
  int seq;
  uint32_t before, total, at = 0, last_at = 0, blocks = 1;
  const auto weight = [&](int s) -> uint32_t {
    const RowShare x = row_share(p, s);
    return x.tiles * x.units;
  };
  const auto place = [&](uint32_t sum) -> uint32_t {
    blocks = row_blocks(p, sum);
    if (blockIdx.x == 0 || blockIdx.x >= blocks) return sum;
    last_at = share_start(blockIdx.x - 1, sum, blocks);
    at = share_start(blockIdx.x, sum, blocks);
    return at;
  };
  RowShare sh = {};
  uint32_t b0 = 0, b1 = 0;
  int head = 0, row = 0;  // the row of the sequence
  bool split = find_share<kRowThreads>(p.seqs.count, weight, place, seq, before, total);
  if (split) {
    sh = row_share(p, seq);
    const uint32_t unit = (at - before) / sh.tiles, start = before + unit * sh.tiles;
    const bool two = sh.rows > p.row_tile;
    head = (int)(two ? unit >> 1 : unit);
    row = (two ? (int)(unit & 1u) * p.row_tile : 0) + r;
    split = start < at && start >= last_at && r < p.row_tile && row < sh.rows;
    b0 = blockIdx.x - 1;
    b1 = share_block(start + sh.tiles - 1, total, blocks);
  }
  // (the first block in any case: a grid that ended before the one ahead of it
  // would let the next one start too early)
  if (!split && (blockIdx.x | blockIdx.y) != 0) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!split) return;
  const int qi = (int)((uint32_t)row / (uint32_t)p.group);
  const int h = head * p.group + row - qi * p.group;
  uint8_t* to = p.out + (sh.span.first_row + qi) * p.o_token + (int64_t)h * p.o_head + 2 * kE * lane;
  float* lse = p.lse ? p.lse + lse_place(sh.span.first_row + qi, p.heads, h) : nullptr;
  float m = ninf, l = 0.0f, acc[kE];
#pragma unroll
  for (int k = 0; k < kE; ++k) acc[k] = 0.0f;
  const int count = (int)(b1 - b0 + 1);
  // partial i of the unit: the first block's is its second (the unit starts
  // there), every other block's its first
  const auto slot = [&](int i) -> int64_t {
    return ((int64_t)(b0 + i) * 2 + (i == 0 ? 1 : 0)) * p.row_tile + r;
  };
  for (int i0 = 0; i0 < count; i0 += 32) {
    // lane: one partial's log-sum-exp
    const float e = i0 + lane < count ? p.row_lse[slot(i0 + lane)] : ninf;
    float mx = e;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    mx = fmaxf(mx, m);
    const float mu = mx == ninf ? 0.0f : mx;
    // roots of the weights; 0 for a part without keys
    const float f = root_ex2(m - mu), wt = root_ex2(e - mu);
    float sum = wt * wt;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    // acc stays the mean of the partials so far: their sum may be too large
    m = mx;
    const float before_l = f * l;
    l = fmaf(f, before_l, sum);
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int k = 0; k < kE; ++k) acc[k] = acc[k] * f * (before_l * inv);
    const int n = min(32, count - i0);
    // (16 partials in flight: with few long units a unit has 20 and more)
    constexpr int kFlight = 16;
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += kFlight) {
      float x[kFlight][kE];
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (k0 + k < n) {
          const float* from = p.row_partials + slot(i0 + k0 + k) * kD + kE * lane;
          if constexpr (kE == 4) {
            const float4 v = *reinterpret_cast<const float4*>(from);
            x[k][0] = v.x;
            x[k][1] = v.y;
            x[k][2] = v.z;
            x[k][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(from);
            x[k][0] = v.x;
            x[k][1] = v.y;
          }
        }
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (k0 + k < n) {
          const float wk = __shfl_sync(0xFFFFFFFFu, wt, k0 + k);
#pragma unroll
          for (int e2 = 0; e2 < kE; ++e2) acc[e2] = fmaf(x[k][e2] * wk, wk * inv, acc[e2]);
        }
    }
  }
#pragma unroll
  for (int k = 0; k < kE; k += 2) st_u32(to + 2 * k, narrow2(acc[k], acc[k + 1], p.half != 0));
  if (lane == 0 && lse)
    *lse = l != 0.0f ? ((m == ninf ? 0.0f : m) + log2f(l)) * 0.69314718055994531f : ninf;
}

// Blocks that fit on an SM (and, once for each device, the kernel's permission
// to use that much shared memory).
template <int kD, int kN, bool kSmallPage>
int rows_per_sm() {
  static int cache[64];
  using K = RowKernel<kD, kN, kSmallPage>;
  const auto kernel = fp8_attention_rows_kernel<kD, kN, kSmallPage>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (cache[dev] == 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (int)K::kBytes) != cudaSuccess) {
    cudaGetLastError();
    return 1;
  }
  return resident_blocks_per_sm(kernel, kRowThreads, K::kBytes, cache);
}

template <int kD, int kN, bool kSmallPage>
int launch(const Fp8AttnParams& p, bool behind_tiles, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.row_grid);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = RowKernel<kD, kN, kSmallPage>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind_tiles ? 1 : 0;
  cudaError_t rc = cudaLaunchKernelEx(&cfg, fp8_attention_rows_kernel<kD, kN, kSmallPage>, p);
  if (rc == cudaSuccess) {
    cfg.gridDim = dim3((unsigned)(p.row_grid + (p.seqs.count + kRowThreads - 1) / kRowThreads),
                       (unsigned)(((p.row_limit < p.row_tile ? p.row_limit : p.row_tile) +
                                   kRowWarps - 1) / kRowWarps));
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    rc = cudaLaunchKernelEx(&cfg, fp8_attention_rows_join_kernel<kD>, p);
  }
  if (rc != cudaSuccess) {
    cudaGetLastError();
    return KVQ_ECUDA;
  }
  return launch_status();
}

}  // namespace

// Blocks of the row kernel on the current device.
int fp8_rows_grid(int64_t head_dim, int row_tile, bool small_page) {
  const int wide = row_tile > 8;
  int per;
  if (head_dim == 128)
    per = small_page ? (wide ? rows_per_sm<128, 2, true>() : rows_per_sm<128, 1, true>())
                     : (wide ? rows_per_sm<128, 2, false>() : rows_per_sm<128, 1, false>());
  else
    per = small_page ? (wide ? rows_per_sm<64, 2, true>() : rows_per_sm<64, 1, true>())
                     : (wide ? rows_per_sm<64, 2, false>() : rows_per_sm<64, 1, false>());
  return per * sm_count();
}

// `behind_tiles`: the tile kernel has just been launched for other sequences of
// the call; this one may start while its last blocks run.
int fp8_rows_launch(const Fp8AttnParams& p, int64_t head_dim, bool behind_tiles,
                    cudaStream_t stream) {
  const bool small = p.cache.page_log2 == 4, wide = p.row_tile > 8;
  if (head_dim == 128)
    return small ? (wide ? launch<128, 2, true>(p, behind_tiles, stream) : launch<128, 1, true>(p, behind_tiles, stream))
                 : (wide ? launch<128, 2, false>(p, behind_tiles, stream) : launch<128, 1, false>(p, behind_tiles, stream));
  return small ? (wide ? launch<64, 2, true>(p, behind_tiles, stream) : launch<64, 1, true>(p, behind_tiles, stream))
               : (wide ? launch<64, 2, false>(p, behind_tiles, stream) : launch<64, 1, false>(p, behind_tiles, stream));
}

}  // namespace kvq
