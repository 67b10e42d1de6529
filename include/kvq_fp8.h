/*
 * kvq_fp8.h — C ABI of the operators around a paged key-value cache with
 * grouped heads held in 8 bits: residual addition + RMSNorm to E4M3, rotation
 * and append of new keys and values, and softmax attention over the pages.
 *
 * The conventions of kvq.h hold (device pointers owned by the caller, nothing
 * allocated, no synchronisation, status codes, host checks before any launch,
 * no device-side value that makes a kernel leave its buffers).
 *
 * The cache. Keys and values are E4M3 codes in pages of page_size tokens
 * (a power of two, 16..256), head h, slot i, element d of page g at byte
 *   g*page_stride + h*head_stride + i*slot_stride + d
 * of k_cache and of v_cache (the same strides for both; all multiples of 16,
 * slot_stride >= head_dim). Every page and head has one power-of-two scale
 * for its keys and one for its values, an E8M0 byte at g*scale_page_stride + h
 * of k_scales and of v_scales: an element stands for code * 2**(byte - 127).
 * Byte 255 (the E8M0 NaN) makes the page's values NaN. block_table[s][j] names
 * the page that holds tokens [j*page_size, (j+1)*page_size) of sequence s; a
 * table_stride of 0 gives all sequences the one row there is. A
 * scale_page_stride of 0, one page's scales for all, is for reading only. What a
 * call writes (the cache in an append, q_out, out) may not overlap itself.
 *
 * Sequences are ragged: the new tokens of sequence s are rows
 * query_start_loc[s] .. query_start_loc[s+1] - 1 of the token-major arrays
 * (non-decreasing; bounds are clamped to [0, num_tokens]). Rows behind the last
 * sequence are neither read nor written.
 */
#ifndef KVQ_FP8_H
#define KVQ_FP8_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KVQ_BF16 0
#define KVQ_FP16 1

/*
 * add_rmsnorm_fp8 — h = x + residual, RMSNorm of h, and its E4M3 codes with
 * binary32 scales (the input of an 8-bit matrix product).
 *
 * Per token, all in binary32:
 *   h = x (+ residual), residual_out = h rounded to the input type,
 *   y = h * (1 / sqrt(mean(h^2) + eps)) * weight   (from the unrounded h),
 * and per group of `group` consecutive values (0: the whole row):
 *   scale = max(largest |y| ignoring NaN, 1e-4) / 448,
 *   code  = E4M3(y / scale) (nearest even, saturating, NaN -> 0x7F).
 *
 * x, residual   bf16 or fp16 (dtype) [num_tokens, hidden], 16-byte aligned
 *               rows (strides in elements, multiples of 8); residual NULL: none
 * residual_out  as x, or NULL; may be x's or residual's own memory (same
 *               stride); needs a residual
 * weight        [hidden], the same type, 16-byte aligned
 * hidden        a multiple of 8, 8..32768; of 128 when group is 128
 * group         0 or 128
 * out           E4M3 codes [num_tokens, hidden], 8-byte aligned rows
 *               (out_stride a multiple of 8)
 * scales        fp32 [num_tokens, hidden/group or 1], row stride scale_stride
 */
int add_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                    const void* weight, float eps, int32_t dtype, int64_t num_tokens,
                    int64_t hidden, int32_t group, uint8_t* out, int64_t out_stride, float* scales,
                    int64_t scale_stride, void* residual_out, int64_t residual_out_stride,
                    cudaStream_t stream);

/*
 * rope_fp8_kv_append — rotate new keys (and, given, queries) by position and
 * append keys and values to their pages.
 *
 * Token i of sequence s (n new tokens) takes cache position p = c + i with
 * c = context_lens[s] clamped to [0, max_pages*page_size]: slot p % page_size
 * of page block_table[s][p / page_size]. Its row r of the cos/sin table is
 * positions[t] (t the token's row), or p when positions is NULL. A token is
 * skipped (nothing of it is read into a scale, written or rotated) when p
 * lies past max_pages*page_size, its page is outside [0, num_pages), or
 * (rotary_dim > 0) r is outside [0, cos_sin_rows); its query is still rotated
 * unless r is outside the table.
 *   Rotation of pair (a, b) with the row's k-th cos and sin, k < rotary_dim/2:
 *   (a*cos - b*sin, b*cos + a*sin) in binary32, each product and sum rounded
 *   separately. interleaved: pairs are elements (2k, 2k+1); otherwise
 *   (k, k + rotary_dim/2). Elements from rotary_dim on are left as they are.
 *   Queries are rounded to their type once.
 *   Page scales. For every page and head that receives tokens, keys and
 *   values apart: amax = max(largest |x| of the new tokens ignoring NaN, 1e-4),
 *   e = ceil(log2(RN(amax * RN(1/448)))), at most 120 (an infinite value then
 *   saturates). If the page already holds earlier tokens of the sequence
 *   (slots below c % page_size of its first page) and its exponent is larger,
 *   that one is kept; if e is larger, the earlier codes are moved to it,
 *   E4M3(code * 2**(old - e)), nearest even. New codes are
 *   E4M3(clamp(x * 2**-e, +-448)), nearest even, NaN -> 0x7F; byte e + 127.
 * Slots that hold neither earlier nor new tokens keep their bytes. No page
 * may receive tokens twice in one call, neither from two sequences nor through
 * two entries of one (the writes would race; a full page may be shared and is
 * not touched).
 *
 * k, v            [num_tokens, num_kv_heads, head_dim] of `dtype`, strides in
 *                 elements (multiples of 8), 16-byte aligned
 * q, q_out        [num_tokens, num_heads, head_dim] likewise; q NULL: none.
 *                 q_out may be q (the same strides)
 * head_dim        a multiple of 16, 16..256
 * cos_sin         fp32 [cos_sin_rows, cos_stride]: rotary_dim/2 cos, then as
 *                 many sin; 16-byte aligned, cos_stride a multiple of 4 and
 *                 >= rotary_dim. NULL when rotary_dim is 0
 * rotary_dim      0 or a multiple of 16, <= head_dim
 * positions       int64 [num_tokens] or NULL
 * block_table     int64 [num_seqs, max_pages], row stride table_stride
 * context_lens    int64 [num_seqs]: tokens in the cache before this call
 * query_start_loc int64 [num_seqs + 1]
 */
int rope_fp8_kv_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                       int64_t v_token_stride, int64_t v_head_stride, const void* q,
                       int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                       int64_t qo_token_stride, int64_t qo_head_stride, int32_t dtype,
                       int64_t num_tokens, int64_t num_heads, int64_t num_kv_heads,
                       int64_t head_dim, const float* cos_sin, int64_t cos_stride,
                       int64_t cos_sin_rows, int64_t rotary_dim, int32_t interleaved,
                       const int64_t* positions, uint8_t* k_cache, uint8_t* v_cache,
                       int64_t num_pages, int64_t page_size, int64_t page_stride,
                       int64_t head_stride, int64_t slot_stride, uint8_t* k_scales,
                       uint8_t* v_scales, int64_t scale_page_stride, const int64_t* block_table,
                       int64_t table_stride, int64_t max_pages, const int64_t* context_lens,
                       const int64_t* query_start_loc, int64_t num_seqs, cudaStream_t stream);

/*
 * fp8_paged_attention — softmax attention of each sequence's new tokens over
 * its keys and values in the cache (which hold the new tokens too).
 *
 * Sequence s has L = seq_lens[s] keys (clamped to [0, max_pages*page_size])
 * and n queries; query i stands at position p = L - n + i. With key head
 * h / (num_heads / num_kv_heads) for head h, over the visible keys j
 *   j < L;  causal: j <= p;  window > 0: j > p - window;  page of j in range,
 *   x_j = sm_scale * q . k_j,  out = sum_j softmax(x)_j v_j (rounded once to
 *   q's type),  lse = log(sum_j exp(x_j)) (natural, fp32).
 * A query without a visible key gets out = 0 and lse = -inf. A key or value
 * that a query does not see never reaches it, whatever bytes its slot holds.
 * Arithmetic: E4M3 codes are exact in fp16; queries enter as fp16 after an
 * exact power-of-two scaling of each row; products accumulate in fp32 on the
 * tensor cores; softmax in fp32; the probabilities, each times its page's value
 * scale, enter the second product as fp16: rounded by 2^-11 of themselves, or,
 * below 2^-22 of the largest such product among the keys that the query sees,
 * by up to 2^-33 of that one. In the normaliser they are not rounded.
 *
 * q, out      [num_tokens, num_heads, head_dim] of `dtype`, strides in
 *             elements (multiples of 8), 16-byte aligned; out may not be q
 * head_dim    64 or 128; num_heads a multiple of num_kv_heads
 * sizes       max_pages * page_size and num_tokens * num_heads / num_kv_heads
 *             below 2**31 - 1024; num_seqs * num_kv_heads *
 *             (max_pages * page_size + 64) at most 2**35
 * max_query_len  at least every n (rows of a longer sequence are unspecified;
 *             0: nothing is read or written)
 * sm_scale    finite, >= 0
 * window      0 (none) or >= 1
 * lse         fp32 [num_tokens, num_heads] or NULL
 * status      device int32 or NULL: set nonzero if an internal wait timed out
 *             (the output is then undefined); never written otherwise
 * workspace   at least fp8_paged_attention_workspace_size(...) bytes of device
 *             memory, 256-byte aligned (never more than 64 MiB, whatever the
 *             shapes). Needs no initialisation; two calls in flight at once
 *             must not share it.
 */
int fp8_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* out,
                        int64_t out_token_stride, int64_t out_head_stride, int32_t dtype,
                        int64_t num_tokens, int64_t num_heads, int64_t num_kv_heads,
                        int64_t head_dim, int64_t max_query_len, const uint8_t* k_cache,
                        const uint8_t* v_cache, int64_t num_pages, int64_t page_size,
                        int64_t page_stride, int64_t head_stride, int64_t slot_stride,
                        const uint8_t* k_scales, const uint8_t* v_scales,
                        int64_t scale_page_stride, const int64_t* block_table,
                        int64_t table_stride, int64_t max_pages, const int64_t* seq_lens,
                        const int64_t* query_start_loc, int64_t num_seqs, float sm_scale,
                        int32_t causal, int64_t window, float* lse, int32_t* status,
                        void* workspace, int64_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes that fp8_paged_attention needs for these shapes on the
 * current device (at most 64 MiB), or KVQ_EINVAL. */
int64_t fp8_paged_attention_workspace_size(int64_t num_seqs, int64_t num_tokens, int64_t num_heads,
                                           int64_t num_kv_heads, int64_t head_dim,
                                           int64_t max_query_len);

/* 1 if a call of these shapes launches a kernel with internal (bounded) waits,
 * whose timing out `status` reports; 0 if there is nothing to report. */
int fp8_paged_attention_waits(int64_t num_tokens, int64_t num_heads, int64_t num_kv_heads,
                              int64_t max_query_len);

/*
 * The three operators with their arguments as 64-bit words: w[0..count-1] are
 * the arguments of the function without `_words`, in its order and without
 * its float and its stream (pointers as integers). For bindings that pay for
 * every argument. count is 15, 39 and 34; any other is KVQ_EINVAL. The words
 * are read before the call returns.
 */
int add_rmsnorm_fp8_words(const int64_t* w, int64_t count, float eps, cudaStream_t stream);
int rope_fp8_kv_append_words(const int64_t* w, int64_t count, cudaStream_t stream);
int fp8_paged_attention_words(const int64_t* w, int64_t count, float sm_scale,
                              cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_FP8_H */
