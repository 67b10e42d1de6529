/*
 * kvq_experts.h — C ABI of the 8-bit matrix products with block scales behind
 * add_rmsnorm_fp8 and fp8_paged_attention, and of a layer of experts around
 * them: routing, the pairs sorted by expert, the experts' products, the
 * weighted sum.
 *
 * The conventions of kvq.h hold (pointers owned by the caller, nothing
 * allocated, no synchronisation, status codes, host checks before any launch,
 * no device-side value that makes a kernel leave its buffers). What a call
 * writes may not overlap itself or what it reads.
 */
#ifndef KVQ_EXPERTS_H
#define KVQ_EXPERTS_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "kvq.h"
#include "kvq_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8_matmul — product of E4M3 rows with E4M3 weights, both with binary32
 * block scales; of one matrix, or of each expert's with its own rows.
 *
 *   out[i][j] = sum over groups g of 128 values:
 *                 a_scales[r][g] * b_scales[e][j / 128][g]
 *                 * sum over the group's l:  a[r][l] * b[e][j][l]
 * rounded once to out's type. The inner sums run on the tensor cores with
 * binary32 accumulators, one for each group; groups are added in binary32.
 *
 *   num_experts 0   one matrix (e = 0), r = i, num_rows = a_rows; offsets and
 *                   rows are NULL
 *   num_experts > 0 out's rows offsets[e] .. offsets[e+1] - 1 belong to expert
 *                   e, r = rows[i], or i where rows is NULL. Offsets are
 *                   clamped to [0, num_rows]; out's rows that no expert has
 *                   are not written, and none is where offsets decrease. A row
 *                   whose r lies outside [0, a_rows) counts as zeros.
 *
 * a          E4M3 [a_rows, k], row stride a_stride, a multiple of 16; 16-byte
 *            aligned, in device memory
 * a_scales   fp32 [a_rows, a_groups], row stride a_scale_stride; a_groups is
 *            ceil(k / 128), or 1: the row's scale
 * b          E4M3 [max(num_experts, 1), n, k]: row stride b_stride and expert
 *            stride b_expert_stride, multiples of 16; 16-byte aligned, in
 *            device memory
 * b_scales   fp32 [max(num_experts, 1), ceil(n / 128), ceil(k / 128)], strides
 *            b_scale_stride and b_scale_expert_stride
 * n, k       1 .. 2**24, k a multiple of 16
 * num_experts  0 .. 1024
 * offsets    int64 [num_experts + 1]
 * rows       int64 [num_rows] or NULL
 * out        bf16 or fp16 (dtype) [num_rows, n], row stride out_stride >= n, in
 *            device memory
 * status     device int32 or NULL: set nonzero if an internal wait timed out
 *            (the output is then undefined); never written otherwise
 * a_rows and num_rows are below 2**31 - 1024; a has a row at least where there
 * are rows to compute. Strides of rows are at most 2**30, of experts 2**39.
 */
int fp8_matmul(const uint8_t* a, int64_t a_stride, const float* a_scales, int64_t a_scale_stride,
               int64_t a_groups, int64_t a_rows, const uint8_t* b, int64_t b_stride,
               int64_t b_expert_stride, const float* b_scales, int64_t b_scale_stride,
               int64_t b_scale_expert_stride, int64_t n, int64_t k, int64_t num_experts,
               const int64_t* offsets, const int64_t* rows, int64_t num_rows, void* out,
               int64_t out_stride, int32_t dtype, int32_t* status, cudaStream_t stream);

/*
 * fp8_gated_matmul — the same product y with 2 * n columns, a gate and an up
 * half, and the activation between them as the input of the next product:
 *
 *   z[i][j] = silu(y[i][j]) * y[i][n + j],  silu(x) = x / (1 + exp(-x)),
 *   scale   = max(largest |z| of the group of 128 ignoring NaN, 1e-4) / 448,
 *   code    = E4M3(z / scale)  (nearest even, saturating, NaN -> 0x7F)
 * in binary32 from the unrounded y. z / scale is formed as z * (448 / largest),
 * within 2^-22 of it; a quotient that near to the middle between two codes may
 * take either. silu is within (9 + 2.35 |x|) 2^-24, relative.
 *
 * b           [max(num_experts, 1), 2 * n, k], b_scales [.., 2 * n / 128, ..]
 * n           a multiple of 128
 * out         E4M3 [num_rows, n], row stride out_stride, a multiple of 16; 16-byte
 *             aligned, in device memory
 * out_scales  fp32 [num_rows, n / 128], row stride out_scale_stride
 */
int fp8_gated_matmul(const uint8_t* a, int64_t a_stride, const float* a_scales,
                     int64_t a_scale_stride, int64_t a_groups, int64_t a_rows, const uint8_t* b,
                     int64_t b_stride, int64_t b_expert_stride, const float* b_scales,
                     int64_t b_scale_stride, int64_t b_scale_expert_stride, int64_t n, int64_t k,
                     int64_t num_experts, const int64_t* offsets, const int64_t* rows,
                     int64_t num_rows, uint8_t* out, int64_t out_stride, float* out_scales,
                     int64_t out_scale_stride, int32_t* status, cudaStream_t stream);

#define KVQ_SOFTMAX 0
#define KVQ_SIGMOID 1
#define KVQ_FP32 2

/*
 * route_experts — scores of the experts for each token, the choice of the best
 * top_k, and their weights.
 *
 * Per token, with x = its logits (NaN counts as -inf, +inf as the largest
 * binary32):
 *   score    softmax(x), or 1 / (1 + exp(-x)); all 0 where every x is -inf
 *   key      score + bias, the sum in binary64; without a bias x itself, which
 *            the scores rise with
 *   groups   > 1: a group is num_experts / groups consecutive experts; its
 *            value is the sum of its two largest score + bias (of score without
 *            a bias), in binary64. The top_groups groups of the largest values
 *            stay, the others' experts are out.
 *   choice   the top_k experts of the largest keys, largest first; equal keys
 *            (and values of groups) go to the lower index
 *   weight   the expert's score, divided by the chosen scores' sum if
 *            renormalize (0 where that is 0), times scale; in binary32, or in
 *            binary64 and rounded once where a chosen score is below 2^-100
 *            (of a score below 2^-1022 what binary64 holds, or nothing)
 * Keys and values that binary32 cannot tell apart are computed in binary64
 * (and what rounding there leaves in doubt, 2^-52, may go either way).
 *
 * logits   bf16, fp16 or fp32 (dtype) [num_tokens, num_experts], row stride
 *          logit_stride
 * bias     fp32 [num_experts] or NULL; -inf puts an expert behind all others,
 *          with NaN or +inf any experts are chosen
 * num_experts  1 .. 1024, a multiple of groups, at least 2 in a group if groups
 *          > 1
 * top_k    1 .. 32, at most the experts of top_groups groups
 * groups   1 .. 32, top_groups 1 .. groups
 * scale    finite
 * experts  int64 [num_tokens, top_k], weights fp32 likewise, contiguous
 */
int route_experts(const void* logits, int64_t logit_stride, int32_t dtype, int64_t num_tokens,
                  int64_t num_experts, int64_t top_k, int32_t score, const float* bias,
                  int64_t groups, int64_t top_groups, int32_t renormalize, float scale,
                  int64_t* experts, float* weights, cudaStream_t stream);

/*
 * sort_by_expert — pairs (token t, choice j) sorted by their expert, pairs of
 * one expert by token and choice.
 *
 *   offsets[e] .. offsets[e+1] - 1   the places of expert e's pairs
 *   rows[i]                          the token of place i
 *   places[t][j]                     the place of the pair, -1 where
 *                                    experts[t][j] lies outside [0, num_experts)
 * Pairs outside have no place: rows[i] of i >= offsets[num_experts] is -1.
 *
 * experts  int64 [num_tokens, top_k], contiguous; num_tokens * top_k below 2**31 - 1024
 * num_experts  1 .. 1024
 * offsets  int64 [num_experts + 1], rows int64 [num_tokens * top_k], places
 *          int64 [num_tokens, top_k]
 * workspace  at least sort_by_expert_workspace_size(...) bytes of device memory
 *          (at most 1 MiB; 0, and then NULL, for few pairs), 4-byte aligned.
 *          Needs no initialisation; two calls in flight at once must not share it.
 */
int sort_by_expert(const int64_t* experts, int64_t num_tokens, int64_t top_k, int64_t num_experts,
                   int64_t* offsets, int64_t* rows, int64_t* places, void* workspace,
                   int64_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes that sort_by_expert needs for these shapes, or KVQ_EINVAL. */
int64_t sort_by_expert_workspace_size(int64_t num_tokens, int64_t top_k, int64_t num_experts);

/*
 * combine_experts — each token's rows of the experts' last product, weighted
 * and added up:
 *   out[t] = base[t] + sum over j of weights[t][j] * y[places[t][j]]
 * in binary32, j ascending, base last, rounded once. A place outside [0, num_rows) adds
 * nothing, whatever its weight.
 *
 * y        bf16 or fp16 (dtype) [num_rows, n], row stride y_stride
 * places   int64 [num_tokens, top_k], weights fp32 likewise, contiguous
 * base     as out, or NULL (nothing); may be out itself
 * out      [num_tokens, n] of the same type
 * n        a multiple of 8; strides multiples of 8, rows 16-byte aligned
 * top_k    1 .. 32
 */
int combine_experts(const void* y, int64_t y_stride, int64_t num_rows, const int64_t* places,
                    const float* weights, int64_t num_tokens, int64_t top_k, const void* base,
                    int64_t base_stride, void* out, int64_t out_stride, int64_t n, int32_t dtype,
                    cudaStream_t stream);

/*
 * The operators with their arguments as 64-bit words: w[0..count-1] are the
 * arguments of the function without `_words`, in its order and without its
 * float and its stream (pointers as integers). count is 22, 23, 13, 9 and 13;
 * any other is KVQ_EINVAL. The words are read before the call returns.
 */
int fp8_matmul_words(const int64_t* w, int64_t count, cudaStream_t stream);
int fp8_gated_matmul_words(const int64_t* w, int64_t count, cudaStream_t stream);
int route_experts_words(const int64_t* w, int64_t count, float scale, cudaStream_t stream);
int sort_by_expert_words(const int64_t* w, int64_t count, cudaStream_t stream);
int combine_experts_words(const int64_t* w, int64_t count, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_EXPERTS_H */
