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
// Every code is used by one thread only when keys are the rows (M) of the
// first product and value elements the rows of the second, with the query
// rows as the 8 columns (N) of mma.m16n8k16: so codes go from global memory
// straight into the registers that need them, with no shared memory and no
// barrier in the loop, and are widened there, E4M3 to fp16 exactly, two per
// instruction. The order of the summed dimension is free, so a thread's 16
// consecutive key elements serve as its fragments; values are paired over two
// tokens by one byte permute. Scores turn from the first product's result
// layout into the second's operand layout by movmatrix.
//
// A warp takes tiles of 32 keys on its own (its own running maximum, sums and
// output), loading the next tile's keys as soon as the scores have consumed
// this one's, and its values after the second product. All (sequence, key
// head) units' tiles are shared out evenly over one resident grid, whatever
// the lengths: a block's warps join their results of a unit in shared memory,
// and units that span blocks are joined by a second kernel from at most two
// partials a block.
#include "fp8_attention.cuh"

namespace kvq {
namespace {

// Global loads issued where they stand: the next tile's loads must not sink
// to their first use.
__device__ __forceinline__ uint4 ld_codes16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ld_codes8(const uint8_t* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
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
  static constexpr int kPart = kD + 1;  // floats of a row of a partial: output, log-sum-exp

  struct Page {
    int64_t g[2];  // page of each half of the tile, -1: none
  };

  static __device__ __forceinline__ Page pages(const Fp8AttnParams& p, int64_t s, int64_t tile,
                                               int64_t keys) {
    Page r;
    const int64_t token = tile * kRowTokens;
    r.g[0] = token < keys ? page_of(p.cache, s, token) : -1;
    r.g[1] = kSmallPage ? (token + 16 < keys ? page_of(p.cache, s, token + 16) : -1) : r.g[0];
    return r;
  }

  struct Keys {
    uint4 c[2][2][kH];  // half, row g / g + 8, piece
    uint32_t scale[2];
  };
  struct Values {
    uint32_t c[2][4][kI / 2];  // half, token, words of kI / 2 * 4 elements
    uint32_t scale[2];
  };

  static __device__ __forceinline__ int64_t half_base(const Fp8AttnParams& p, const Page& pg,
                                                      int64_t tile, int head, int h) {
    const int64_t slot = (tile * kRowTokens + 16 * h) & (((int64_t)1 << p.cache.page_log2) - 1);
    return pg.g[h] * p.cache.page_stride + head * p.cache.head_stride + slot * p.cache.slot_stride;
  }

  static __device__ __forceinline__ void load_keys(const Fp8AttnParams& p, const Page& pg,
                                                   int64_t tile, int head, int off, Keys& k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (pg.g[h] >= 0) {
        const uint8_t* at = p.cache.k + half_base(p, pg, tile, head, h) + off;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kH; ++i)
            k.c[h][r][i] = ld_codes16(at + (int64_t)(8 * r) * p.cache.slot_stride + 64 * i);
        k.scale[h] = ld_byte(p.cache.k_scales + pg.g[h] * p.cache.scale_page_stride + head);
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kH; ++i) k.c[h][r][i] = make_uint4(0, 0, 0, 0);
        k.scale[h] = 127;
      }
    }
  }

  static __device__ __forceinline__ void load_values(const Fp8AttnParams& p, const Page& pg,
                                                     int64_t tile, int head, int off, Values& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (pg.g[h] >= 0) {
        const uint8_t* at = p.cache.v + half_base(p, pg, tile, head, h) + off;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* row = at + (int64_t)((r & 1) + 8 * (r >> 1)) * p.cache.slot_stride;
          if constexpr (kD == 128) {
            const uint4 x = ld_codes16(row);
            v.c[h][r][0] = x.x;
            v.c[h][r][1] = x.y;
            v.c[h][r][2] = x.z;
            v.c[h][r][3] = x.w;
          } else {
            const uint2 x = ld_codes8(row);
            v.c[h][r][0] = x.x;
            v.c[h][r][1] = x.y;
          }
        }
        v.scale[h] = ld_byte(p.cache.v_scales + pg.g[h] * p.cache.scale_page_stride + head);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < kI / 2; ++i) v.c[h][r][i] = 0;
        v.scale[h] = 127;
      }
    }
  }
};

template <int kD, int kN, bool kSmallPage>
__global__ void __launch_bounds__(kRowThreads) fp8_attention_rows_kernel(const Fp8AttnParams p) {
  using K = RowKernel<kD, kN, kSmallPage>;
  constexpr int kH = K::kH, kI = K::kI, kRows = K::kRows;
  __shared__ float sm_o[kRowWarps][kRows][kD + 4];
  __shared__ float sm_m[kRowWarps][kRows], sm_l[kRowWarps][kRows], sm_v[kRowWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const float ninf = neg_inf();

  // this block's share [at, end) of all tiles
  int seq;
  int64_t before, total;
  const auto weight = [&](int s) -> int64_t {
    const RowShare r = row_share(p, s);
    return r.tiles * r.row_tiles * p.kv_heads;
  };
  // the total first: the share's start depends on it
  find_share<kRowThreads>(p.seqs.count, -1, weight, seq, before, total);
  if (total == 0) return;
  const int64_t blocks = row_blocks(p, total);
  if ((int64_t)blockIdx.x >= blocks) return;
  int64_t at = share_start(blockIdx.x, total, blocks);
  const int64_t end = share_start(blockIdx.x + 1, total, blocks);
  __syncthreads();
  find_share<kRowThreads>(p.seqs.count, at, weight, seq, before, total);

  while (at < end) {
    // the unit that holds tile `at`
    RowShare sh = row_share(p, seq);
    const int64_t share = sh.tiles * sh.row_tiles * p.kv_heads;
    if (at >= before + share) {
      before += share;
      ++seq;
      continue;
    }
    const int64_t unit = (at - before) / sh.tiles;
    const int64_t unit_start = before + unit * sh.tiles;
    const int64_t seg_end = min(end, unit_start + sh.tiles);
    const int head = (int)(unit / sh.row_tiles);
    const int row0 = (int)(unit - (int64_t)head * sh.row_tiles) * kRows;
    const int rows = (int)min((int64_t)kRows, sh.n * p.group - row0);
    const int64_t tile0 = sh.first + (at - unit_start), tile1 = sh.first + (seg_end - unit_start);

    // query fragments: row 8 c + g, as fp16 times a power of two that brings
    // the row's largest magnitude to [2**14, 2**15)
    uint32_t qf[kN][kH][4][2];
    float qs[kN][2];                // per result column: scale_log2 / that power
    int32_t lim[kN][2], low[kN][2];  // visible keys [low, lim) of the column's row, from key 0
    // (positions are at most 2**40: keys are addressed relative to tile0)
    const int64_t base_key = tile0 * kRowTokens;
    const bool half = p.half != 0;
    int32_t all_lim = 0x7FFFFFFF, all_low = 0;
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const int r = row0 + 8 * c + g;
      const bool have = 8 * c + g < rows;
      const int qi = have ? r / p.group : 0;
      const uint8_t* qrow = p.q + (sh.first_row + qi) * p.q_token +
                            (int64_t)(head * p.group + (have ? r - qi * p.group : 0)) * p.q_head;
      uint4 w[kH][2];
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[i][j] = have ? ld_nc_v4(qrow + 2 * (64 * i + 16 * t + 8 * j)) : make_uint4(0, 0, 0, 0);
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[8];
          widen8(w[i][j], half, f);
#pragma unroll
          for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // amax in [2**e, 2**(e + 1)); scaled by 2**(14 - e)
      const int e = amax > 0.0f ? max((int)(__float_as_uint(amax) >> 23), 16) - 127 : 0;
      const float up = __uint_as_float((uint32_t)(min(14 - e, 127) + 127) << 23);
      const float down = p.scale_log2 / up;
#pragma unroll
      for (int i = 0; i < kH; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[8];
          widen8(w[i][j], half, f);
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
        const int64_t qi2 = col < rows ? (row0 + col) / p.group : 0;
        int64_t lo, hi;
        key_range(p, sh.keys, sh.n, qi2, qi2 + 1, lo, hi);
        lim[c][j] = (int32_t)clamp64(hi - base_key, 0, 0x7FFFFFFF);
        low[c][j] = (int32_t)clamp64(lo - base_key, 0, 0x7FFFFFFF);
        all_lim = min(all_lim, lim[c][j]);
        all_low = max(all_low, low[c][j]);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      all_lim = min(all_lim, __shfl_xor_sync(0xFFFFFFFFu, all_lim, o));
      all_low = max(all_low, __shfl_xor_sync(0xFFFFFFFFu, all_low, o));
    }

    float m[kN][2], l[kN][2], o[kI][kN][4];
    float vref = ninf;
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      m[c][0] = m[c][1] = ninf;
      l[c][0] = l[c][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kI; ++i) o[i][c][0] = o[i][c][1] = o[i][c][2] = o[i][c][3] = 0.0f;
    }

    const int k_off = g * p.cache.slot_stride + 16 * t;
    const int v_off = 2 * t * p.cache.slot_stride + (kD / 8) * g;
    int64_t tile = tile0 + warp;
    typename K::Page pg = K::pages(p, seq, tile, tile < tile1 ? sh.keys : 0);
    typename K::Page pg_next = K::pages(p, seq, tile + kRowWarps, tile + kRowWarps < tile1 ? sh.keys : 0);
    typename K::Keys kk;
    typename K::Values vv;
    K::load_keys(p, pg, tile, head, k_off, kk);
    K::load_values(p, pg, tile, head, v_off, vv);
    for (; tile < tile1; tile += kRowWarps) {
      // scores: two halves of 16 keys x 8 kN rows
      float s[2][kN][4];
      float ks[2] = {e8m0_value(kk.scale[0]), e8m0_value(kk.scale[1])};
      const bool page_ok[2] = {pg.g[0] >= 0, pg.g[1] >= 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < kN; ++c) s[h][c][0] = s[h][c][1] = s[h][c][2] = s[h][c][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kH; ++i) {
          const uint32_t a[4] = {kk.c[h][0][i].x, kk.c[h][0][i].y, kk.c[h][0][i].z, kk.c[h][0][i].w};
          const uint32_t b[4] = {kk.c[h][1][i].x, kk.c[h][1][i].y, kk.c[h][1][i].z, kk.c[h][1][i].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(a[w] & 0xFFFFu), a2 = e4m3x2_to_f16x2(a[w] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(b[w] & 0xFFFFu), a3 = e4m3x2_to_f16x2(b[w] >> 16);
#pragma unroll
            for (int c = 0; c < kN; ++c)
              mma_f16(s[h][c], a0, a1, a2, a3, qf[c][i][w][0], qf[c][i][w][1]);
          }
        }
      }
      // the next tile's keys
      const int64_t next = tile + kRowWarps;
      pg = pg_next;
      pg_next = K::pages(p, seq, next + kRowWarps, next + kRowWarps < tile1 ? sh.keys : 0);
      K::load_keys(p, pg, next, head, k_off, kk);

      // scaled scores; -inf where a row does not see the key
      const int32_t key0 = (int32_t)((tile - tile0) * kRowTokens);
      const bool whole = page_ok[0] && page_ok[1] && key0 + kRowTokens <= all_lim && key0 >= all_low;
      float top[kN][2];
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[c][j] = ninf;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float x = s[h][c][2 * r + j] * (qs[c][j] * ks[h]);
              if (!whole) {
                const int32_t key = key0 + 16 * h + 8 * r + g;
                if (!page_ok[h] || key >= lim[c][j] || key < low[c][j]) x = ninf;
              }
              s[h][c][2 * r + j] = x;
              top[c][j] = fmaxf(top[c][j], x);
            }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1)
            top[c][j] = fmaxf(top[c][j], __shfl_xor_sync(0xFFFFFFFFu, top[c][j], d));
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (vv.scale[h] == 255u) {  // the page's values are NaN
          vv.scale[h] = 127u;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < kI / 2; ++i) vv.c[h][r][i] = 0x7F7F7F7Fu;
        }
      // references: rescale the sums when a row's maximum or the value scale
      // has outgrown them
      const float ve[2] = {e8m0_log2(vv.scale[0]), e8m0_log2(vv.scale[1])};
      float vtop = ninf;
      if (page_ok[0]) vtop = ve[0];
      if (page_ok[1]) vtop = fmaxf(vtop, ve[1]);
      bool grow = vtop > vref + kVLagLog2;
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) grow |= top[c][j] > m[c][j] + kLagLog2;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        float vf = 1.0f;
        if (vtop > vref + kVLagLog2) {
          vf = ex2(vref - vtop);  // 0 the first time
          vref = vtop;
        }
#pragma unroll
        for (int c = 0; c < kN; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float f = 1.0f;
            if (top[c][j] > m[c][j]) {
              f = ex2(m[c][j] - top[c][j]);
              m[c][j] = top[c][j];
            }
            l[c][j] *= f;
            f *= vf;
#pragma unroll
            for (int i = 0; i < kI; ++i) {
              o[i][c][j] *= f;
              o[i][c][2 + j] *= f;
            }
          }
      }
      // probabilities times 2**(kPLog2 + value exponent - reference)
      uint32_t pf[2][kN][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float dv = page_ok[h] ? fmaxf(ve[h] - vref, kVFloorLog2) : 0.0f;
        const float back = ex2(-dv);
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          float pr[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float shift = dv + kPLog2 - (m[c][j] == ninf ? 0.0f : m[c][j]);
            pr[j] = ex2(s[h][c][j] + shift);
            pr[2 + j] = ex2(s[h][c][2 + j] + shift);
            l[c][j] = fmaf(pr[j] + pr[2 + j], back, l[c][j]);
          }
          // results are keys x rows, (row g, columns 2t, 2t + 1); the second
          // product wants (rows 2t, 2t + 1, column g)
          pf[h][c][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
          pf[h][c][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
        }
      }
      // values of keys that no row sees must not reach the product, where
      // 0 * NaN is NaN; a NaN that only some rows see is added to them below
      if (!whole) {
        const int32_t end_key = (int32_t)clamp64(sh.keys - base_key, 0, 0x7FFFFFFF);
        bool found = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int32_t key = key0 + 16 * h + 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
            for (int i = 0; i < kI / 2; ++i) {
              if (key >= end_key) vv.c[h][r][i] = 0;
              found |= has_nan_code(vv.c[h][r][i]);
            }
          }
        if (__any_sync(0xFFFFFFFFu, found)) {
          // a rare path: for every token of the tile, the quad's owner says
          // which of its elements are NaN, and the quad marks the rows that
          // see it; then the codes are cleared
#pragma unroll 1
          for (int k = 0; k < 32; ++k) {
            const int owner = (k & 7) >> 1, h = k >> 4, r = (k & 1) + 2 * ((k >> 3) & 1);
            uint32_t bad = 0;
            if (owner == t) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int rr = 0; rr < 4; ++rr)
                  if (hh == h && rr == r) {
#pragma unroll
                    for (int i = 0; i < kI / 2; ++i) {
                      const uint32_t ok = number_codes(vv.c[hh][rr][i]);
#pragma unroll
                      for (int b = 0; b < 4; ++b)
                        if (((ok >> (8 * b)) & 1u) == 0u) bad |= 1u << (4 * i + b);
                    }
                  }
            }
            bad = __shfl_sync(0xFFFFFFFFu, bad, (lane & ~3) | owner);
            const int32_t key = key0 + k;
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
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int i = 0; i < kI / 2; ++i) vv.c[h][r][i] &= number_codes(vv.c[h][r][i]);
        }
      }
      // output += V^T P^T: block i holds elements (kD / 8) g + 2 i (+ 1)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int w = 0; w < kI / 2; ++w) {
          const uint32_t x = prmt(vv.c[h][0][w], vv.c[h][1][w], 0x5140);
          const uint32_t y = prmt(vv.c[h][2][w], vv.c[h][3][w], 0x5140);
          const uint32_t x2 = prmt(vv.c[h][0][w], vv.c[h][1][w], 0x7362);
          const uint32_t y2 = prmt(vv.c[h][2][w], vv.c[h][3][w], 0x7362);
          const uint32_t a0 = e4m3x2_to_f16x2(x & 0xFFFFu), a1 = e4m3x2_to_f16x2(x >> 16);
          const uint32_t a2 = e4m3x2_to_f16x2(y & 0xFFFFu), a3 = e4m3x2_to_f16x2(y >> 16);
          const uint32_t b0 = e4m3x2_to_f16x2(x2 & 0xFFFFu), b1 = e4m3x2_to_f16x2(x2 >> 16);
          const uint32_t b2 = e4m3x2_to_f16x2(y2 & 0xFFFFu), b3 = e4m3x2_to_f16x2(y2 >> 16);
#pragma unroll
          for (int c = 0; c < kN; ++c) {
            mma_f16(o[2 * w][c], a0, a1, a2, a3, pf[h][c][0], pf[h][c][1]);
            mma_f16(o[2 * w + 1][c], b0, b1, b2, b3, pf[h][c][0], pf[h][c][1]);
          }
        }
      K::load_values(p, pg, next, head, v_off, vv);
    }

    // join the block's warps
#pragma unroll
    for (int c = 0; c < kN; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[c][j] += __shfl_xor_sync(0xFFFFFFFFu, l[c][j], d);
        const int col = 8 * c + 2 * t + j;
        if (g == 0) {
          sm_m[warp][col] = m[c][j];
          sm_l[warp][col] = l[c][j];
        }
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          sm_o[warp][col][(kD / 8) * g + 2 * i] = o[i][c][j];
          sm_o[warp][col][(kD / 8) * g + 2 * i + 1] = o[i][c][2 + j];
        }
      }
    if (lane == 0) sm_v[warp] = vref;
    __syncthreads();
    const bool complete = at == unit_start && seg_end == unit_start + sh.tiles;
    float* part = p.row_partials +
                  ((int64_t)blockIdx.x * 2 + (at == unit_start ? 1 : 0)) * kRows * K::kPart;
    // thread: 4 elements of a row
    for (int id = threadIdx.x; id < rows * (kD / 4); id += kRowThreads) {
      const int r = id / (kD / 4), d = 4 * (id - r * (kD / 4));
      float mx = ninf;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) mx = fmaxf(mx, sm_m[w][r]);
      if (mx == ninf) mx = 0.0f;
      // a row without keys has sum 0; one whose scores are all NaN has
      // maximum -inf and a NaN sum, which stays
      float sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float f = ex2(sm_m[w][r] - mx);
        sum = fmaf(sm_l[w][r], f, sum);
        const float fv = f * exp2f(sm_v[w]);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = fmaf(sm_o[w][r][d + k], fv, acc[k]);
      }
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
      const float lse2 = sum != 0.0f ? mx + log2f(sum) - kPLog2 : ninf;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] *= inv;
      if (complete) {
        const int qi = (row0 + r) / p.group;
        const int h = head * p.group + (row0 + r) - qi * p.group;
        uint8_t* to = p.out + (sh.first_row + qi) * p.o_token + (int64_t)h * p.o_head + 2 * d;
        st_v2(to, narrow2(acc[0], acc[1], half), narrow2(acc[2], acc[3], half));
        if (d == 0 && p.lse)
          p.lse[(sh.first_row + qi) * p.heads + h] = lse2 * 0.69314718055994531f;
      } else {
        float* to = part + r * K::kPart;
#pragma unroll
        for (int k = 0; k < 4; ++k) to[d + k] = acc[k];
        if (d == 0) to[kD] = lse2;
      }
    }
    __syncthreads();
    at = seg_end;
  }
}

// Joins the partials of every unit that spans blocks, and writes zeros for
// units without a key. Block: a sequence and one of its units.
template <int kD>
__global__ void __launch_bounds__(kRowThreads) fp8_attention_rows_join_kernel(const Fp8AttnParams p) {
  constexpr int kPart = kD + 1;
  const float ninf = neg_inf();
  const int seq = blockIdx.x;
  const RowShare sh = row_share(p, seq);
  if (sh.row_tiles == 0) return;
  int unused;
  int64_t unused_before, total, before = 0;
  const auto weight = [&](int s) -> int64_t {
    const RowShare r = row_share(p, s);
    return r.tiles * r.row_tiles * p.kv_heads;
  };
  const auto weight_before = [&](int s) -> int64_t { return s < seq ? weight(s) : 0; };
  find_share<kRowThreads>(p.seqs.count, -1, weight_before, unused, unused_before, before);
  __syncthreads();
  find_share<kRowThreads>(p.seqs.count, -1, weight, unused, unused_before, total);
  const int64_t blocks = total ? row_blocks(p, total) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t unit = blockIdx.y; unit < (int64_t)sh.row_tiles * p.kv_heads; unit += gridDim.y) {
    const int64_t u0 = before + unit * sh.tiles, u1 = u0 + sh.tiles;
    int64_t b0 = 0, b1 = 0;
    if (sh.tiles) {
      b0 = share_block(u0, total, blocks);
      b1 = share_block(u1 - 1, total, blocks);
      if (b0 == b1) continue;  // written whole
    }
    const int head = (int)(unit / sh.row_tiles);
    const int row0 = (int)(unit - (int64_t)head * sh.row_tiles) * p.row_tile;
    const int rows = (int)min((int64_t)p.row_tile, sh.n * p.group - row0);
    for (int id = threadIdx.x; id < rows * (kD / 4); id += kRowThreads) {
      const int r = id / (kD / 4), d = 4 * (id - r * (kD / 4));
      float mx = ninf, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (sh.tiles) {
        const auto slot = [&](int64_t b) {
          const int64_t start = share_start(b, total, blocks);
          return p.row_partials +
                 ((b * 2 + (start <= u0 ? 1 : 0)) * p.row_tile + r) * (int64_t)kPart;
        };
        for (int64_t b = b0; b <= b1; ++b) mx = fmaxf(mx, slot(b)[kD]);
        if (mx == ninf) mx = 0.0f;
        for (int64_t b = b0; b <= b1; ++b) {
          const float* from = slot(b);
          const float f = ex2(from[kD] - mx);  // 0 for a part without keys
          sum += f;
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[k] = fmaf(from[d + k], f, acc[k]);
        }
      }
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
      const int qi = (row0 + r) / p.group;
      const int h = head * p.group + (row0 + r) - qi * p.group;
      uint8_t* to = p.out + (sh.first_row + qi) * p.o_token + (int64_t)h * p.o_head + 2 * d;
      st_v2(to, narrow2(acc[0] * inv, acc[1] * inv, p.half != 0),
            narrow2(acc[2] * inv, acc[3] * inv, p.half != 0));
      if (d == 0 && p.lse)
        p.lse[(sh.first_row + qi) * p.heads + h] =
            sum != 0.0f ? (mx + log2f(sum)) * 0.69314718055994531f : ninf;
    }
  }
}

template <int kD, int kN, bool kSmallPage>
int rows_per_sm() {
  static int cache[64];
  return resident_blocks_per_sm(fp8_attention_rows_kernel<kD, kN, kSmallPage>, kRowThreads, 0,
                                cache);
}

template <int kD, int kN, bool kSmallPage>
int launch(const Fp8AttnParams& p, cudaStream_t stream) {
  fp8_attention_rows_kernel<kD, kN, kSmallPage><<<(unsigned)p.row_grid, kRowThreads, 0, stream>>>(p);
  const int rc = launch_status();
  if (rc != KVQ_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  const int64_t units = ((int64_t)p.row_limit + p.row_tile - 1) / p.row_tile * p.kv_heads;
  cfg.gridDim = dim3((unsigned)p.seqs.count, (unsigned)(units < 65535 ? units : 65535));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fp8_attention_rows_join_kernel<kD>, p) != cudaSuccess) {
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

int fp8_rows_launch(const Fp8AttnParams& p, int64_t head_dim, cudaStream_t stream) {
  const bool small = p.cache.page_log2 == 4, wide = p.row_tile > 8;
  if (head_dim == 128)
    return small ? (wide ? launch<128, 2, true>(p, stream) : launch<128, 1, true>(p, stream))
                 : (wide ? launch<128, 2, false>(p, stream) : launch<128, 1, false>(p, stream));
  return small ? (wide ? launch<64, 2, true>(p, stream) : launch<64, 1, true>(p, stream))
               : (wide ? launch<64, 2, false>(p, stream) : launch<64, 1, false>(p, stream));
}

}  // namespace kvq
