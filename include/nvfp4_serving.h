/*
 * nvfp4_serving.h - C ABI of the operators of one decoding step over NVFP4
 * data, in libmoe_nvfp4.so next to the calls of moe_nvfp4.h:
 *
 *   kv_block_tables        pages and slots of a paged cache from the requests'
 *                          lengths, on the GPU
 *   nvfp4_paged_attention  attention over the paged NVFP4 key/value cache that
 *                          nvfp4_quantize_paged writes
 *   moe_layer_nvfp4,       a whole mixture-of-experts layer for a few tokens,
 *   moe_layer_bf16         from the router's logits to the summed output
 *
 * Formats, status codes, memory and stream rules are those of moe_nvfp4.h:
 * every pointer is a device pointer, the caller owns every buffer (workspaces
 * included), the library allocates nothing, keeps nothing between calls and
 * never synchronizes, arguments are checked on the host before any HIP call,
 * inputs and outputs must not overlap. A workspace holds nothing between
 * calls; two calls that may run at the same time need one each. No call uses
 * atomics on memory: the same inputs give the same bytes.
 */
#ifndef NVFP4_SERVING_H
#define NVFP4_SERVING_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Block tables and slot maps of a paged cache. Request b holds
 * c = context_lens[b] tokens in the cache and brings n = query_lens[b] new
 * ones (negative lengths count as 0; context_lens NULL: all 0). The cache is
 * made of pages of page_size slots; page p holds slots p * page_size up to
 * (p + 1) * page_size - 1, and token t of request b stands in page
 * block_table[b][t / page_size].
 *   New pages: the request's first ceil(c / page_size) entries are there
 *   already; entries from there to ceil((c + n) / page_size) - 1 are taken
 *   from free_pages, in the order of the requests and of their pages,
 *   starting at free_pages[free_begin[0]] (free_begin NULL: 0), and written
 *   to block_table (-1 where the list has no more). No other entry is
 *   written. free_end[0] = free_begin[0] + the number of pages wanted: more
 *   than num_free tells that the list was too short.
 *   num_free == -1: no list, no page is taken, every entry is there already
 *   (num_free == 0 is an empty list). With it,
 *   context_lens NULL and query_lens the lengths of whole requests this
 *   gives the slots of all their tokens (for nvfp4_dequantize_paged).
 *   Outputs: query_offsets[b] = the new tokens before request b
 *   (num_seqs + 1 entries); seq_lens[b] = c + n; slots[query_offsets[b] + i] =
 *   the slot of request b's i-th new token, -1 where its table entry is
 *   negative or past max_pages (nvfp4_quantize_paged skips such a token);
 *   slots from query_offsets[num_seqs] up to max_tokens are -1. Tokens past
 *   max_tokens get no slot; sums saturate at 2^31 - 1. A page past max_pages
 *   is not taken.
 * block_table [num_seqs][ld_table] int32, max_pages columns used;
 * free_begin[0] outside [0, num_free] counts as an empty list and is taken as
 * 0 in free_end. query_offsets, seq_lens, free_end and slots are all
 * required. No output (block_table among them, the columns used) may share
 * memory with an input or another output; such a call is refused with
 * NVFP4_ERROR_INVALID_VALUE.
 * num_seqs <= 4096, max_tokens < 2^31, page_size >= 1. num_seqs == 0 is no
 * error: the outputs are written. One kernel.
 */
nvfp4_status_t kv_block_tables(const int32_t *context_lens, const int32_t *query_lens,
                               int64_t num_seqs, int32_t page_size,
                               const int32_t *free_pages, int64_t num_free,
                               const int32_t *free_begin, int32_t *block_table,
                               int64_t ld_table, int64_t max_pages,
                               int32_t *query_offsets, int32_t *seq_lens,
                               int64_t *slots, int64_t max_tokens, int32_t *free_end,
                               hipStream_t stream);

/*
 * Attention over the paged NVFP4 cache. Request b has n = query_offsets[b+1] -
 * query_offsets[b] query rows (q rows query_offsets[b] ...) and
 * L = seq_lens[b] tokens in the cache, the new ones included: its i-th query
 * stands at position p = L - n + i. With g = heads / kv_heads, query head h
 * reads key/value head h / g:
 *   s_j = scale * k_gs * sum_d q[d] * k_j[d]   (k_j: E2M1 code times E4M3 scale)
 *   for the tokens j with 0 <= j < L, j <= p when causal, j > p - window when
 *   window > 0, whose page is inside the cache (a table entry outside
 *   [0, num_slots / page_size) or past max_pages hides its tokens);
 *   out = v_gs * sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), m = max s_j,
 *   lse = m + ln sum_j exp(s_j - m)            (FP32, natural logarithm).
 * A row that sees no token gets out = 0 and lse = -inf.
 *   q       [tokens][ld_q] BF16, heads * head_dim columns used
 *   caches  k_packed, v_packed [num_slots][kv_heads * head_dim / 2] and
 *           k_scales, v_scales [num_slots][kv_heads * head_dim / 16], as
 *           nvfp4_quantize_paged writes them (num_slots a multiple of
 *           page_size); k_gs, v_gs: NULL (1.0) or one FP32 value each
 *   block_table [num_seqs][ld_table] int32, max_pages columns used
 *   seq_lens [num_seqs], query_offsets [num_seqs + 1] int32, as
 *           kv_block_tables writes them; a length below 0 counts as 0, one
 *           past max_pages * page_size as that
 *   out     [tokens][ld_out] BF16, heads * head_dim columns; lse
 *           [tokens][heads] FP32 or NULL. Rows of no request (in front of
 *           query_offsets[0], behind query_offsets[num_seqs]) keep their
 *           values.
 *   max_query_len, max_seq_len: the largest n and L that the caller expects.
 *           They choose the kernel and the split of the work, not the result:
 *           longer requests are computed too, only slower. A max_seq_len far
 *           above the real lengths costs workgroups without work, time in
 *           the join and workspace, which grow with it up to 256 splits.
 *   workspace: nvfp4_paged_attention_workspace(...) bytes (may be 0, then
 *           workspace may be NULL), 16-byte aligned.
 * Products are exact products of the BF16 q and the NVFP4 values, summed in
 * FP32; a query row is scaled by a power of two into FP16's range, where its
 * values are exact down to 2^-31 of the row's largest and smaller ones are
 * off by at most 2^-39 of that. Probabilities are rounded to FP16 for the
 * product with v: off by at most 2^-11 relative, or by 2^-36 of the row's
 * largest probability where that is more (so a tail of n tokens is off by at
 * most n 2^-36 of that). Sums are FP32. q, the global scales and the scales
 * of a request's L tokens must be finite (nvfp4_quantize_paged writes no
 * others from finite values); a NaN in k_gs or in a row of q makes out and
 * lse NaN in the rows that it reaches. Slots that no row can see (behind L,
 * of hidden pages, of no request) may hold anything. head_dim is 64, 128 or
 * 256; heads a multiple of kv_heads, at most 1024; ld_q, ld_out multiples of
 * 8; q, out, packed caches 16-byte aligned, scale caches 4-byte (8 for
 * head_dim 128, 16 for 256); num_slots < 2^31, tokens * heads <= 2^30,
 * num_seqs <= 65535, num_seqs * kv_heads <= 2^22, max_pages * page_size <=
 * 2^30; window >= 2^31 hides nothing. One kernel, or two where a long
 * context is split over workgroups.
 */
nvfp4_status_t nvfp4_paged_attention(const uint16_t *q, int64_t tokens, int64_t ld_q,
                                     int32_t heads, int32_t kv_heads, int32_t head_dim,
                                     const uint8_t *k_packed, const uint8_t *k_scales,
                                     const uint8_t *v_packed, const uint8_t *v_scales,
                                     int64_t num_slots, int32_t page_size,
                                     const int32_t *block_table, int64_t ld_table,
                                     int64_t max_pages, const int32_t *seq_lens,
                                     const int32_t *query_offsets, int64_t num_seqs,
                                     int64_t max_query_len, int64_t max_seq_len,
                                     float scale, int32_t causal, int64_t window,
                                     const float *k_gs, const float *v_gs, uint16_t *out,
                                     int64_t ld_out, float *lse, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that nvfp4_paged_attention needs for these sizes (the
 * same arguments as the call's), or -1 where the call refuses them. Needs no
 * GPU. */
int64_t nvfp4_paged_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                        int32_t head_dim, int64_t num_seqs,
                                        int64_t max_query_len, int64_t max_seq_len,
                                        int64_t window);

/*
 * A whole mixture-of-experts layer for a few tokens (1 to 64):
 *   ids[t] = the top_k experts with the largest logits[t][e], in descending
 *            order, ties to the lower expert; a logit that is NaN or -inf
 *            leaves its expert out (id -1, weight 0 where fewer than top_k
 *            are left);
 *   w[t][k] = softmax(logits[t])[ids[t][k]], or with renormalize != 0 the
 *            softmax over the chosen logits alone;
 *   a = x[t] W1[e]^T with interleaved [gate x8, up x8, ...] columns as in
 *            moe_l1_gemm_swiglu_nvfp4, h = silu(gate) * up in FP32;
 *   out[t] = sum_k w[t][k] * (h W2[e]^T), rounded to BF16 once.
 * x [tokens][ld_x] BF16; logits [tokens][num_experts] FP32; out
 * [tokens][ld_out] BF16, hidden columns; topk_ids [tokens][top_k] int32,
 * topk_weights [tokens][top_k] FP32 (both written).
 * moe_layer_bf16:  w1 [E][2*inter][hidden], w2 [E][hidden][inter] BF16.
 * moe_layer_nvfp4: the same matrices as nvfp4_quantize writes them: packed
 *   codes [..][cols / 2], scales [..][cols / 16] and a global scale per
 *   expert (gs1, gs2 [E], NULL: 1.0), cols along the summed axis.
 * Every product is exact and sums are FP32. The activations of both products
 * (x, then h in FP32) are brought to the matrix instructions' types:
 *   NVFP4 weights: each token's values in a run of the summed axis (256 or 512
 *   for x, 256 for h) are scaled by a power of two into FP16's range; x keeps
 *   every bit down to 2^-31 of the largest value of its run, smaller values are
 *   off by at most 2^-39 of that; h is rounded, by 2^-11 relative or by 2^-39 of
 *   the largest value of its run where that is more;
 *   BF16 weights: x as it is, h as the sum of two BF16 numbers (2^-17 relative).
 * x must be finite, and h inside the BF16 range: a token's row of out is infinite
 * or NaN otherwise; other tokens' rows are not touched by it.
 * hidden and inter are multiples of 32, at least 32, at most 2^20;
 * num_experts <= 512; top_k <= 32 and <= num_experts; tokens * top_k * inter * 4
 * and the bytes that x spans ((tokens - 1) * ld_x + hidden, times 2) below
 * 2^31 - 4096; ld_x, ld_out multiples of 8. x, out, packed codes, BF16 weights
 * and workspace are 16-byte aligned, scales 2-byte, logits, gs, ids and
 * topk_weights 4-byte. tokens == 0 is a no-op. workspace:
 * moe_layer_workspace(...) bytes. Three kernels.
 */
nvfp4_status_t moe_layer_nvfp4(const uint16_t *x, int64_t tokens, int64_t ld_x,
                               const float *logits, const uint8_t *w1_packed,
                               const uint8_t *w1_scales, const float *gs1,
                               const uint8_t *w2_packed, const uint8_t *w2_scales,
                               const float *gs2, int64_t hidden, int64_t inter,
                               int32_t num_experts, int32_t top_k, int32_t renormalize,
                               uint16_t *out, int64_t ld_out, int32_t *topk_ids,
                               float *topk_weights, void *workspace,
                               int64_t workspace_bytes, hipStream_t stream);

nvfp4_status_t moe_layer_bf16(const uint16_t *x, int64_t tokens, int64_t ld_x,
                              const float *logits, const uint16_t *w1, const uint16_t *w2,
                              int64_t hidden, int64_t inter, int32_t num_experts,
                              int32_t top_k, int32_t renormalize, uint16_t *out,
                              int64_t ld_out, int32_t *topk_ids, float *topk_weights,
                              void *workspace, int64_t workspace_bytes,
                              hipStream_t stream);

/* Bytes of workspace of the two calls above, or -1 where they refuse these
 * sizes. Needs no GPU. */
int64_t moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter,
                            int32_t num_experts, int32_t top_k);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_SERVING_H */
