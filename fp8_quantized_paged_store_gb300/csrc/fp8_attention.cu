// fp8_attention.cu — fp8_paged_attention: argument checks, workspace and the
// choice of kernels.
#include "fp8_attention.cuh"

namespace kvq {
int fp8_rows_grid(int64_t head_dim, int row_tile, bool small_page);
int fp8_rows_launch(const Fp8AttnParams& p, int64_t head_dim, bool behind_tiles,
                    cudaStream_t stream);
int64_t fp8_tiles_workspace(int64_t units, int64_t kv_heads, int chunks, int64_t head_dim);
int fp8_tiles_launch(const Fp8AttnParams& p, int64_t head_dim, cudaStream_t stream);

namespace {

bool shapes_ok(int64_t num_seqs, int64_t num_tokens, int64_t num_heads, int64_t num_kv_heads,
               int64_t head_dim, int64_t max_query_len) {
  return num_seqs >= 0 && num_seqs <= (int64_t)1 << 20 && num_tokens >= 0 &&
         num_tokens <= (int64_t)1 << 30 && num_kv_heads >= 1 && num_heads >= num_kv_heads &&
         num_heads <= 65535 && num_heads % num_kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128) && max_query_len >= 0;
}

// Which kernels a call launches, and how its workspace is laid out. The host
// knows the longest run of new tokens but not the lengths, so a call whose
// longest run takes the tile kernel launches the row kernel too, for the
// sequences with few rows, unless all runs must be equally long.
struct Plan {
  bool rows, tiles;
  int row_limit, row_tile, row_grid, tile_chunks;
  int64_t tile_units, row_bytes, bytes;
};

Plan plan_for(int64_t num_seqs, int64_t num_tokens, int64_t num_heads, int64_t num_kv_heads,
              int64_t head_dim, int64_t max_query_len, bool small_page) {
  Plan r = {};
  const int64_t group = num_heads / num_kv_heads;
  const int64_t longest = max_query_len < num_tokens ? max_query_len : num_tokens;
  r.tiles = longest > kFewRows / group;
  r.rows = group <= kFewRows && (!r.tiles || num_seqs > num_tokens / longest);
  if (r.rows) {
    r.row_limit = r.tiles ? kFewRows : (int)(group * longest);
    r.row_tile = r.row_limit > 8 ? 16 : 8;
    r.row_grid = fp8_rows_grid(head_dim, r.row_tile, small_page);
    r.row_bytes = ((int64_t)r.row_grid * 2 * r.row_tile * (head_dim + 1) * 4 + 255) / 256 * 256;
  }
  if (r.tiles) {
    r.tile_units = num_tokens * group / 256 + num_seqs;
    const int64_t parts = sm_count() / (r.tile_units * num_kv_heads);
    r.tile_chunks = (int)(parts < 1 ? 1 : (parts > 16 ? 16 : parts));
  }
  r.bytes = r.row_bytes +
            (r.tiles ? fp8_tiles_workspace(r.tile_units, num_kv_heads, r.tile_chunks, head_dim) : 0);
  return r;
}

}  // namespace
}  // namespace kvq

extern "C" int64_t fp8_paged_attention_workspace_size(int64_t num_seqs, int64_t num_tokens,
                                                      int64_t num_heads, int64_t num_kv_heads,
                                                      int64_t head_dim, int64_t max_query_len) {
  using namespace kvq;
  if (!shapes_ok(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_query_len))
    return KVQ_EINVAL;
  if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return 0;
  const int64_t a = plan_for(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                             max_query_len, false).bytes;
  const int64_t b = plan_for(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                             max_query_len, true).bytes;
  return a > b ? a : b;
}

extern "C" int fp8_paged_attention(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, void* out,
    int64_t out_token_stride, int64_t out_head_stride, int32_t dtype, int64_t num_tokens,
    int64_t num_heads, int64_t num_kv_heads, int64_t head_dim, int64_t max_query_len,
    const uint8_t* k_cache, const uint8_t* v_cache, int64_t num_pages, int64_t page_size,
    int64_t page_stride, int64_t head_stride, int64_t slot_stride, const uint8_t* k_scales,
    const uint8_t* v_scales, int64_t scale_page_stride, const int64_t* block_table,
    int64_t table_stride, int64_t max_pages, const int64_t* seq_lens,
    const int64_t* query_start_loc, int64_t num_seqs, float sm_scale, int32_t causal,
    int64_t window, float* lse, int32_t* status, void* workspace, int64_t workspace_bytes,
    cudaStream_t stream) {
  using namespace kvq;
  if (!shapes_ok(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_query_len) ||
      (dtype != KVQ_BF16 && dtype != KVQ_FP16) || (causal != 0 && causal != 1) || window < 0)
    return KVQ_EINVAL;
  if (!(sm_scale >= 0.0f) || sm_scale > 3.0e38f / 1.5f) return KVQ_EINVAL;
  Fp8AttnParams p = {};
  if (!fp8_cache_params(const_cast<uint8_t*>(k_cache), const_cast<uint8_t*>(v_cache), num_pages,
                        page_size, page_stride, head_stride, slot_stride,
                        const_cast<uint8_t*>(k_scales), const_cast<uint8_t*>(v_scales),
                        scale_page_stride, block_table, table_stride, max_pages, num_seqs,
                        num_kv_heads, head_dim, false, p.cache))
    return KVQ_EINVAL;
  // rows, keys, and the tiles of all key heads of all sequences stay
  // countable in 31 bits
  if (num_tokens * (num_heads / num_kv_heads) > 0x7FFFFFFF - 1024 ||
      max_pages > (0x7FFFFFFF - 1024) / page_size)
    return KVQ_EINVAL;
  if (num_seqs > 0 && max_pages * page_size + 64 > ((int64_t)1 << 35) / num_kv_heads / num_seqs)
    return KVQ_EINVAL;
  const int64_t cap = INT64_MAX / 16 / (num_tokens + 1);
  auto bad = [&](int64_t token, int64_t head) {
    return token < 0 || head < 0 || token % 8 || head % 8 || token > cap ||
           head > INT64_MAX / 16 / num_heads;
  };
  if (bad(q_token_stride, q_head_stride) || bad(out_token_stride, out_head_stride))
    return KVQ_EINVAL;
  if (!runs_apart<2>(head_dim, {num_tokens, num_heads}, {out_token_stride, out_head_stride}))
    return KVQ_EINVAL;
  if (num_tokens == 0 || num_seqs == 0 || max_query_len == 0) return KVQ_OK;
  if (!q || !out || q == out || !k_cache || !v_cache || !k_scales || !v_scales || !seq_lens ||
      !query_start_loc || (max_pages > 0 && !block_table))
    return KVQ_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 8) || !aligned(seq_lens, 8) || !aligned(query_start_loc, 8) ||
      !aligned(lse, 4) || !aligned(status, 4) || !aligned(workspace, 256))
    return KVQ_EINVAL;
  const Plan plan = plan_for(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                             max_query_len, page_size == 16);
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return KVQ_EINVAL;
  if (plan.tile_units * num_kv_heads * plan.tile_chunks > 0x7FFFFFFF) return KVQ_EINVAL;
  p.seqs = {query_start_loc, seq_lens, num_tokens, (int32_t)num_seqs};
  p.q = static_cast<const uint8_t*>(q);
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.status = status;
  p.q_token = 2 * q_token_stride;
  p.q_head = 2 * q_head_stride;
  p.o_token = 2 * out_token_stride;
  p.o_head = 2 * out_head_stride;
  p.window = window;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.heads = (int32_t)num_heads;
  p.kv_heads = (int32_t)num_kv_heads;
  p.group = (int32_t)(num_heads / num_kv_heads);
  p.causal = causal;
  p.half = dtype == KVQ_FP16;
  p.row_limit = plan.row_limit;  // 0: the tile kernel takes every sequence
  p.row_tile = plan.row_tile;
  p.row_grid = plan.row_grid;
  p.row_partials = static_cast<float*>(workspace);
  p.row_lse = p.row_partials + (int64_t)plan.row_grid * 2 * plan.row_tile * head_dim;
  p.tile_units = plan.tile_units;
  p.tile_chunks = plan.tile_chunks;
  p.tile_partials =
      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.row_bytes);
  if (plan.tiles) {
    const int rc = fp8_tiles_launch(p, head_dim, stream);
    if (rc != KVQ_OK) return rc;
  }
  if (!plan.rows) return KVQ_OK;
  return fp8_rows_launch(p, head_dim, plan.tiles, stream);
}

extern "C" int fp8_paged_attention_waits(int64_t num_tokens, int64_t num_heads,
                                         int64_t num_kv_heads, int64_t max_query_len) {
  if (num_kv_heads < 1 || num_heads < num_kv_heads) return 0;
  const int64_t longest = max_query_len < num_tokens ? max_query_len : num_tokens;
  return longest > kvq::kFewRows / (num_heads / num_kv_heads) ? 1 : 0;
}
