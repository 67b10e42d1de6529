// fp8_append.cu — rope_fp8_kv_append: rotate new keys and queries by position
// and append keys and values to the pages of an E4M3 cache with one
// power-of-two scale for each page and head.
//
//   (a, b) -> (a cos - b sin, b cos + a sin), every product and sum rounded
//   separately;  e = max(old exponent, ceil(log2(max(amax, 1e-4) / 448)));
//   code = E4M3(x * 2**-e).
//
// Bound by memory: 2 bytes read and 1 written per key and value element, 2
// and 2 per query element.
//
// An item is one (page, head, keys or values). It belongs to one team of 1 to
// 8 warps, so no two teams write one page and head: no atomics, and the result
// does not depend on any order. The team's threads load and rotate the page's
// new rows once, keep them in registers, agree on the largest magnitude, and
// write the codes. A thread's unit is 16 elements, the two runs of 8 that the
// rotation pairs with each other (neighbours when interleaved, half a rotary
// width apart otherwise), so a rotation needs no other lane.
// All items of the call, heads within pages within sequences, are shared
// evenly by the teams of one resident grid: a team loads its next item's rows
// while it writes the last one's codes, and keeps cos and sin in shared memory
// for all heads of a page.
// Blocks past those rotate queries: a warp takes a token, each lane one unit
// of several heads, with its cos and sin kept in registers; the first loads go
// out before the token's sequence is searched.
//
// Seven chunks of 300 to 2048 tokens, 32 heads on 8 key heads of 128: 37 us,
// 5260 GB/s (78 % of a copy's rate). The pages' share, a quarter of the bytes,
// is bound by an item's chain (load, maximum, barrier, store): reading the rows
// twice, a block to a page, took 56 us in all, one pass without even shares 47
// us. Three blocks an SM (80 registers) spill: 45 us.
#include "fp8_cache.cuh"

namespace kvq {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kHold = 2;   // units a thread of a team keeps
constexpr int kQSteps = 4; // query units a lane loads at once

struct AppendParams {
  Fp8Cache cache;
  Fp8Seqs seqs;  // lens: tokens in the cache before
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* q;
  uint8_t* q_out;
  int64_t k_token, k_head, v_token, v_head;      // bytes
  int64_t q_token, q_head, qo_token, qo_head;    // bytes
  const float* cos_sin;
  int64_t cos_stride, cos_rows;
  const int64_t* positions;
  int32_t page_blocks;  // blocks of page work; the rest rotate queries
  int32_t team_log2;    // warps of a team
  int32_t lanes_log2;   // lanes of a row: `units`, rounded up to a power of two
  int32_t heads, kv_heads;
  int32_t units;        // head_dim / 16
  int32_t rot_units;    // rotary_dim / 16
};

// First elements of a unit's two runs of 8.
template <bool kInter>
__device__ __forceinline__ void unit_runs(const AppendParams& p, int u, int& a, int& b) {
  if (!kInter && u < p.rot_units) {
    a = 8 * u;
    b = 8 * p.rot_units + 8 * u;
  } else {
    a = 16 * u;
    b = 16 * u + 8;
  }
}

__device__ __forceinline__ uint4 ld_row16(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// 16 bytes into shared memory, complete after cp.async.wait_all.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}

__device__ __forceinline__ void unpack8(float4 a, float4 b, float (&f)[8]) {
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// cos and sin of the 8 pairs of unit u < rot_units of a table row.
__device__ __forceinline__ void load_angles(const AppendParams& p, int64_t row, int u,
                                            float (&c)[8], float (&s)[8]) {
  const float* at = p.cos_sin + row * p.cos_stride + 8 * u;
  const float4 c0 = ld_f4(at), c1 = ld_f4(at + 4);
  const float* st = at + 8 * p.rot_units;
  const float4 s0 = ld_f4(st), s1 = ld_f4(st + 4);
  c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
  c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
  s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
  s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
}

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
  b = y;
}

template <bool kInter>
__device__ __forceinline__ void rotate_unit(float (&x)[8], float (&y)[8], const float (&c)[8],
                                            const float (&s)[8]) {
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
      rotate_pair(y[2 * i], y[2 * i + 1], c[i + 4], s[i + 4]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(x[i], y[i], c[i], s[i]);
  }
}

// Row of the cos/sin table for token row t at cache position pos, or -1.
__device__ __forceinline__ int64_t table_row(const AppendParams& p, int64_t t, int64_t pos) {
  if (p.rot_units == 0) return 0;
  const int64_t r = p.positions ? p.positions[t] : pos;
  return (uint64_t)r < (uint64_t)p.cos_rows ? r : -1;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
  return make_uint2(cvt_e4m3x2(f[0] * inv, f[1] * inv) | (cvt_e4m3x2(f[2] * inv, f[3] * inv) << 16),
                    cvt_e4m3x2(f[4] * inv, f[5] * inv) | (cvt_e4m3x2(f[6] * inv, f[7] * inv) << 16));
}

// Four codes moved to a larger exponent: E4M3(code * f), f = 2**(old - new).
__device__ __forceinline__ uint32_t move_codes(uint32_t w, float f) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(w, lo, hi);
  const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
  return cvt_e4m3x2(a.x * f, a.y * f) | (cvt_e4m3x2(b.x * f, b.y * f) << 16);
}

// Pages that n new tokens behind ctx earlier ones touch.
__device__ __forceinline__ int64_t touched_pages(const AppendParams& p, int64_t n, int64_t ctx) {
  return n ? ((ctx + n - 1) >> p.cache.page_log2) - (ctx >> p.cache.page_log2) + 1 : 0;
}

// Largest value over a team (as ordered bits: none is NaN, and -1 is the only
// negative one). Also a barrier of the team; successive calls take turns with
// `slots`.
__device__ __forceinline__ float team_max(float v, int team_log2, int* slots) {
  int bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_int(v));
  if (team_log2 > 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) slots[warp] = bits;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (warp >> team_log2)), "r"(32 << team_log2)
                 : "memory");
    bits = __reduce_max_sync(0xFFFFFFFFu, slots[(warp >> team_log2 << team_log2) +
                                                (lane & ((1 << team_log2) - 1))]);
  }
  return __int_as_float(bits);
}

// Items [item, end) of the call, by one team. The item lies at or after
// sequence s, before which `before` pages are touched.
template <bool kHalf, bool kInter>
__device__ __forceinline__ void append_items(const AppendParams& p, int s, int64_t before,
                                             int64_t item, int64_t end) {
  __shared__ int slots[2][kAppendWarps];
  // cos and sin of a thread's units, its own places alone (in registers, with
  // 100 bytes spilled, ragged chunks took 40 us instead of 37)
  __shared__ float4 angles[4 * kHold][kAppendThreads];
  // A row is taken by 2**lanes_log2 lanes (the lanes past its units idle), and
  // a thread takes the same unit of `step` rows further down, kHold times.
  const int me = threadIdx.x & ((32 << p.team_log2) - 1);
  const int u = me & ((1 << p.lanes_log2) - 1), i0 = me >> p.lanes_log2;
  const int step = (32 << p.team_log2) >> p.lanes_log2;
  const int round = kHold * step;
  const int subs = 2 * p.kv_heads;
  int a, b;
  unit_runs<kInter>(p, u, a, b);
  const bool turns = u < p.rot_units;
  int64_t ordinal = item / subs;  // of the page among the touched ones
  int sub = (int)(item - ordinal * subs);
  int64_t first = 0, n = 0, ctx = 0, pages = -1;
  // the page that `load` reads for
  int64_t page, t0, pos0;
  int kept, count;
  bool fresh;  // its first item
  const auto enter_page = [&]() {
    while (pages < 0 || ordinal >= before + pages) {
      if (pages >= 0) {
        before += pages;
        ++s;
      }
      seq_rows(p.seqs, s, first, n);
      ctx = clamp64(p.seqs.lens[s], 0, p.cache.capacity);
      pages = touched_pages(p, n, ctx);
    }
    const int64_t column = (ctx >> p.cache.page_log2) + (ordinal - before);
    const int64_t start = column << p.cache.page_log2;
    pos0 = ctx > start ? ctx : start;  // first new token in the page
    kept = (int)(pos0 - start);        // earlier tokens of the sequence
    t0 = first + (pos0 - ctx);
    page = -1;
    count = 0;
    if (start < p.cache.capacity) {
      page = page_of(p.cache, s, start);
      count = (int)min(ctx + n - pos0, (int64_t)(1 << p.cache.page_log2) - kept);
    }
    fresh = true;
  };
  const auto last_round = [&]() { return count > round ? (count - 1) / round * round : 0; };
  uint4 w0[kHold], w1[kHold];
  float x[kHold][8], y[kHold][8];
  bool got[kHold];  // false past the end and for a skipped token
  // The units of the round at row `at`: into w0 and w1; for a page's first
  // keys, and in every round of a page with several, also the angles.
  const auto load = [&](int at) {
    const bool keys = sub < p.kv_heads;
    const int64_t stride = keys ? p.k_token : p.v_token;
    const uint8_t* from = keys ? p.k + sub * p.k_head : p.v + (sub - p.kv_heads) * p.v_head;
    from += (t0 + (at + i0)) * stride;
    const bool look = fresh || count > round;
    fresh = false;
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      const int i = at + i0 + h * step;
      if (look) got[h] = u < p.units && i < count;
      if (got[h]) {
        w0[h] = ld_row16(from + 2 * a);
        w1[h] = ld_row16(from + 2 * b);
      }
      from += step * stride;
      if (look && got[h]) {
        const int64_t row = table_row(p, t0 + i, pos0 + i);
        got[h] = row >= 0;
        if (keys && turns && got[h]) {
          const float* from_row = p.cos_sin + row * p.cos_stride + 8 * u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            copy16(&angles[4 * h + k][threadIdx.x],
                   from_row + 4 * (k & 1) + (k >> 1) * 8 * p.rot_units);
        }
      }
    }
  };
  const auto widen_and_turn = [&](bool keys) {
    const bool turn = keys && turns;
    if (turn) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      if (!got[h]) continue;
      widen8(w0[h], kHalf, x[h]);
      widen8(w1[h], kHalf, y[h]);
      if (turn) {
        float c[8], sn[8];
        unpack8(angles[4 * h][threadIdx.x], angles[4 * h + 1][threadIdx.x], c);
        unpack8(angles[4 * h + 2][threadIdx.x], angles[4 * h + 3][threadIdx.x], sn);
        rotate_unit<kInter>(x[h], y[h], c, sn);
      }
    }
  };
  enter_page();
  load(last_round());
#pragma unroll 1
  for (; item < end; ++item) {
    const bool keys = sub < p.kv_heads;
    const int head = keys ? sub : sub - p.kv_heads;
    const int now_kept = kept, now_count = count;
    const int64_t now_page = page;
    uint8_t* scale = (keys ? p.cache.k_scales : p.cache.v_scales) +
                     now_page * p.cache.scale_page_stride + head;
    const int old = now_kept > 0 && now_page >= 0 ? (int)*scale - 127 : 0;
    // the last round first: the first one's units stay in registers
    float amax = -1.0f;
    int at = last_round();
#pragma unroll 1
    while (true) {
      widen_and_turn(keys);
#pragma unroll
      for (int h = 0; h < kHold; ++h) {
        if (!got[h]) continue;
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fmaxf(fabsf(x[h][k]), fabsf(y[h][k])));
        amax = fmaxf(amax, top);
      }
      if (at == 0) break;
      at -= round;
      load(at);
    }
    bool mine[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) mine[h] = got[h];
    const auto next = [&]() {
      if (item + 1 < end) {
        if (++sub == subs) {
          sub = 0;
          ++ordinal;
          enter_page();
        }
        load(last_round());
      }
    };
    const bool one_round = now_count <= round;
    if (one_round) next();
    amax = team_max(amax, p.team_log2, slots[item & 1]);  // also: the team has read the scale
    if (amax >= 0.0f && now_page >= 0) {  // (not every token skipped)
      uint8_t* codes = (keys ? p.cache.k : p.cache.v) + now_page * p.cache.page_stride +
                       head * p.cache.head_stride;
      int e = ceil_pow2_exponent(__fmul_rn(fmaxf(amax, 1e-4f), 1.0f / 448.0f));
      e = min(e, 120);
      if (now_kept > 0) {
        if (old >= e) {
          e = old;
        } else if (u < p.units) {
          const int diff = e - old;  // at most 247: two exact powers
          const float f1 = exp2_neg(min(diff, 126)), f2 = exp2_neg(max(diff - 126, 0));
#pragma unroll 1
          for (int i = i0; i < now_kept; i += step) {
            uint8_t* to = codes + (int64_t)i * p.cache.slot_stride + 16 * u;
            uint4 w = ld_row16(to);
            w = make_uint4(move_codes(w.x, f1), move_codes(w.y, f1), move_codes(w.z, f1),
                           move_codes(w.w, f1));
            if (diff > 126)
              w = make_uint4(move_codes(w.x, f2), move_codes(w.y, f2), move_codes(w.z, f2),
                             move_codes(w.w, f2));
            st_v4(to, w);
          }
        }
      }
      if (me == 0) *scale = (uint8_t)(e + 127);
      const float inv = exp2_neg(e);
#pragma unroll 1
      for (int r = 0; r < now_count; r += round) {
        if (r > 0) {
          load(r);
          widen_and_turn(keys);
#pragma unroll
          for (int h = 0; h < kHold; ++h) mine[h] = got[h];
        }
        uint8_t* to = codes + (int64_t)(now_kept + r + i0) * p.cache.slot_stride;
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
          if (mine[h]) {
            const uint2 cx = codes8(x[h], inv), cy = codes8(y[h], inv);
            if (kInter || !turns) {
              st_v4(to + a, make_uint4(cx.x, cx.y, cy.x, cy.y));
            } else {
              st_v2(to + a, cx.x, cx.y);
              st_v2(to + b, cy.x, cy.y);
            }
          }
          to += step * p.cache.slot_stride;
        }
      }
    }
    if (!one_round) next();
  }
}

// Sequence of token row t, found by a warp: the number of sequences that end
// at or before it, from 32 of their (non-decreasing) ends at a time. -1 past
// the last one.
__device__ __forceinline__ int seq_of(const Fp8Seqs& q, int64_t t) {
  const int lane = threadIdx.x & 31;
  int before = 0, left = q.count;
#pragma unroll 1
  while (left > 0) {
    const int step = (left + 31) / 32;
    const int probe = (lane + 1) * step;  // of `left`, from 1 on
    const bool ends = probe <= left && clamp64(q.start[before + probe], 0, q.num_tokens) <= t;
    const int passed = __popc(__ballot_sync(0xFFFFFFFFu, ends)) * step;
    before += passed;
    // the next probe's run, without the probe itself unless it was past the end
    left = step == 1 ? 0 : min(left - passed, step - 1);
  }
  return before < q.count ? before : -1;
}

template <bool kHalf, bool kInter>
__device__ __forceinline__ void rotate_query(const AppendParams& p, int64_t t) {
  const int lane = threadIdx.x & 31;
  const int per_step = 32 >> p.lanes_log2;  // heads a warp takes at once (>= 2)
  const int sub = lane >> p.lanes_log2, u = lane & ((1 << p.lanes_log2) - 1);
  int a, b;
  unit_runs<kInter>(p, u, a, b);
  const uint8_t* from = p.q + t * p.q_token;
  uint8_t* to = p.q_out + t * p.qo_token;
  const int heads = u < p.units ? p.heads : 0;
  uint4 w0[kQSteps], w1[kQSteps];
  const auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kQSteps; ++i) {
      const int h = h0 + i * per_step;
      if (h < heads) {
        w0[i] = ld_row16(from + h * p.q_head + 2 * a);
        w1[i] = ld_row16(from + h * p.q_head + 2 * b);
      }
    }
  };
  load(sub);
  const int s = seq_of(p.seqs, t);
  if (s < 0) return;
  int64_t first, n;
  seq_rows(p.seqs, s, first, n);
  if (t < first) return;  // in no sequence (before the first one's start)
  const int64_t ctx = clamp64(p.seqs.lens[s], 0, p.cache.capacity);
  const int64_t row = table_row(p, t, ctx + (t - first));
  if (row < 0) return;
  float c[8], sn[8];
  const bool turn = u < p.rot_units;
  if (turn) load_angles(p, row, u, c, sn);
#pragma unroll 1
  for (int h0 = sub; h0 < heads; h0 += kQSteps * per_step) {
    if (h0 != sub) load(h0);
#pragma unroll
    for (int i = 0; i < kQSteps; ++i) {
      const int h = h0 + i * per_step;
      if (h >= heads) break;
      if (turn) {
        float x[8], y[8];
        widen8(w0[i], kHalf, x);
        widen8(w1[i], kHalf, y);
        rotate_unit<kInter>(x, y, c, sn);
        w0[i] = narrow8(x, kHalf);
        w1[i] = narrow8(y, kHalf);
      }
      st_v4(to + h * p.qo_head + 2 * a, w0[i]);
      st_v4(to + h * p.qo_head + 2 * b, w1[i]);
    }
  }
}

template <bool kHalf, bool kInter>
__global__ void __launch_bounds__(kAppendThreads, 2) fp8_append_kernel(const AppendParams p) {
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x >= p.page_blocks) {
    const int64_t t = (int64_t)(blockIdx.x - p.page_blocks) * kAppendWarps + warp;
    if (t < p.seqs.num_tokens) rotate_query<kHalf, kInter>(p, t);
    return;
  }
  const int teams = kAppendWarps >> p.team_log2;
  const int64_t subs = 2 * p.kv_heads;
  int64_t share = 0;  // items of a team
  const auto touched = [&](int s) -> int64_t {
    int64_t first, n;
    seq_rows(p.seqs, s, first, n);
    return touched_pages(p, n, clamp64(p.seqs.lens[s], 0, p.cache.capacity));
  };
  const auto first_page = [&](int64_t total) -> int64_t {
    const int64_t all = (int64_t)p.page_blocks * teams;
    share = (total * subs + all - 1) / all;
    return blockIdx.x * teams * share / subs;
  };
  int s;
  int64_t before, total;
  if (!find_share<kAppendThreads>(p.seqs.count, touched, first_page, s, before, total)) return;
  const int64_t item = ((int64_t)blockIdx.x * teams + (warp >> p.team_log2)) * share;
  const int64_t end = min(item + share, total * subs);
  if (item < end) append_items<kHalf, kInter>(p, s, before, item, end);
}

}  // namespace
}  // namespace kvq

extern "C" int rope_fp8_kv_append(
    const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
    int64_t v_token_stride, int64_t v_head_stride, const void* q, int64_t q_token_stride,
    int64_t q_head_stride, void* q_out, int64_t qo_token_stride, int64_t qo_head_stride,
    int32_t dtype, int64_t num_tokens, int64_t num_heads, int64_t num_kv_heads, int64_t head_dim,
    const float* cos_sin, int64_t cos_stride, int64_t cos_sin_rows, int64_t rotary_dim,
    int32_t interleaved, const int64_t* positions, uint8_t* k_cache, uint8_t* v_cache,
    int64_t num_pages, int64_t page_size, int64_t page_stride, int64_t head_stride,
    int64_t slot_stride, uint8_t* k_scales, uint8_t* v_scales, int64_t scale_page_stride,
    const int64_t* block_table, int64_t table_stride, int64_t max_pages,
    const int64_t* context_lens, const int64_t* query_start_loc, int64_t num_seqs,
    cudaStream_t stream) {
  using namespace kvq;
  if (num_tokens < 0 || num_tokens > (int64_t)1 << 30 || num_seqs < 0 ||
      num_seqs > (int64_t)1 << 20 || (dtype != KVQ_BF16 && dtype != KVQ_FP16) ||
      (interleaved != 0 && interleaved != 1))
    return KVQ_EINVAL;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16) return KVQ_EINVAL;
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16) return KVQ_EINVAL;
  AppendParams p;
  if (!fp8_cache_params(k_cache, v_cache, num_pages, page_size, page_stride, head_stride,
                        slot_stride, k_scales, v_scales, scale_page_stride, block_table,
                        table_stride, max_pages, num_seqs, num_kv_heads, head_dim, true, p.cache))
    return KVQ_EINVAL;
  const int64_t cap = INT64_MAX / 16 / (num_tokens + 1);
  auto bad = [&](int64_t token, int64_t head, int64_t heads) {
    return token < 0 || head < 0 || token % 8 || head % 8 || token > cap ||
           head > INT64_MAX / 16 / heads || (heads > 1 && head < head_dim);
  };
  if (bad(k_token_stride, k_head_stride, num_kv_heads) ||
      bad(v_token_stride, v_head_stride, num_kv_heads))
    return KVQ_EINVAL;
  if (q) {
    if (num_heads < 1 || num_heads > 65535 || !q_out ||
        bad(q_token_stride, q_head_stride, num_heads) ||
        bad(qo_token_stride, qo_head_stride, num_heads))
      return KVQ_EINVAL;
    if (q == q_out && (q_token_stride != qo_token_stride || q_head_stride != qo_head_stride))
      return KVQ_EINVAL;
    if (!runs_apart<2>(head_dim, {num_tokens, num_heads}, {qo_token_stride, qo_head_stride}))
      return KVQ_EINVAL;
  }
  if (rotary_dim > 0 && (cos_sin_rows < 1 || cos_stride < rotary_dim || cos_stride % 4 ||
                         cos_stride > INT64_MAX / 16 / cos_sin_rows))
    return KVQ_EINVAL;
  if (num_tokens == 0 || num_seqs == 0) return KVQ_OK;
  if (!k || !v || !k_cache || !v_cache || !k_scales || !v_scales || !context_lens ||
      !query_start_loc || (max_pages > 0 && !block_table) || (rotary_dim > 0 && !cos_sin))
    return KVQ_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cos_sin, 16) ||
      !aligned(positions, 8) || !aligned(block_table, 8) || !aligned(context_lens, 8) ||
      !aligned(query_start_loc, 8))
    return KVQ_EINVAL;
  p.seqs = {query_start_loc, context_lens, num_tokens, (int32_t)num_seqs};
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.q = static_cast<const uint8_t*>(q);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.k_token = 2 * k_token_stride;
  p.k_head = 2 * k_head_stride;
  p.v_token = 2 * v_token_stride;
  p.v_head = 2 * v_head_stride;
  p.q_token = 2 * q_token_stride;
  p.q_head = 2 * q_head_stride;
  p.qo_token = 2 * qo_token_stride;
  p.qo_head = 2 * qo_head_stride;
  p.cos_sin = cos_sin;
  p.cos_stride = cos_stride;
  p.cos_rows = cos_sin_rows;
  p.positions = positions;
  p.heads = (int32_t)(q ? num_heads : 0);
  p.kv_heads = (int32_t)num_kv_heads;
  p.units = (int32_t)(head_dim / 16);
  p.rot_units = (int32_t)(rotary_dim / 16);
  p.lanes_log2 = 0;
  while (1 << p.lanes_log2 < p.units) ++p.lanes_log2;
  // A team is as large as keeps the new rows of a page in its registers, going
  // by the average sequence.
  const int64_t average = (num_tokens + num_seqs - 1) / num_seqs;
  const int64_t page_units = (average < page_size ? average : page_size) << p.lanes_log2;
  p.team_log2 = 0;
  while (p.team_log2 < 3 && (int64_t)kHold * 32 << p.team_log2 < page_units) ++p.team_log2;
  const int64_t teams = kAppendWarps >> p.team_log2;  // of a block
  // Touched pages: a sequence of n > 0 tokens reaches at most
  // (n - 1) / page_size + 2 pages, and no more than n.
  int64_t pages = num_tokens / page_size + 2 * num_seqs;
  if (pages > num_tokens) pages = num_tokens;
  auto* kernel = dtype == KVQ_FP16
                     ? (interleaved ? fp8_append_kernel<true, true> : fp8_append_kernel<true, false>)
                     : (interleaved ? fp8_append_kernel<false, true> : fp8_append_kernel<false, false>);
  p.page_blocks = (int32_t)grid_for((2 * num_kv_heads * pages + teams - 1) / teams, 2);
  const int64_t blocks = p.page_blocks + (q ? (num_tokens + kAppendWarps - 1) / kAppendWarps : 0);
  if (blocks > 0x7FFFFFFF) return KVQ_EINVAL;
  kernel<<<(unsigned)blocks, kAppendThreads, 0, stream>>>(p);
  return launch_status();
}
