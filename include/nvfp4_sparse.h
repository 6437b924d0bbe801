/*
 * nvfp4_sparse.h - C ABI of the operators of sparse attention over the paged
 * NVFP4 key/value cache, in libmoe_nvfp4.so next to the calls of moe_nvfp4.h and
 * nvfp4_serving.h. One step of a model that reads a few pages of a long
 * context runs them in this order, behind kv_block_tables:
 *
 *   nvfp4_rope_append       q and k rotated by their positions, k and v written
 *                           into the cache
 *   nvfp4_page_keys         an 8-bit key for each page that the new tokens complete
 *   nvfp4_select_pages      the pages that each new token attends to, by their keys
 *   nvfp4_sparse_attention  attention over the tokens of the listed pages
 *
 * Formats, status codes, memory and stream rules are those of moe_nvfp4.h:
 * every pointer is a device pointer, the caller owns every buffer (workspaces
 * included), the library allocates nothing, keeps nothing between calls and
 * never synchronizes, arguments are checked on the host before any HIP call,
 * inputs and outputs must not overlap. A workspace holds nothing between
 * calls; two calls that may run at the same time need one each. The same
 * inputs give the same bytes.
 *
 * Requests, as kv_block_tables describes them: request b owns the tokens (rows of
 * q) query_offsets[b] up to query_offsets[b + 1] - 1, n of them, at the end of
 * its L = seq_lens[b] tokens (below 0: 0; past max_pages * page_size: that),
 * its i-th at position L - n + i; token t of the request stands in page
 * block_table[b][t / page_size] of the cache. A page is hidden where its table
 * entry is outside [0, num_slots / page_size). query_offsets do not fall; with some
 * that do, every call ends and keeps to its buffers, lists hold pages of the table,
 * and nothing more is specified.
 */
#ifndef NVFP4_SPARSE_H
#define NVFP4_SPARSE_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotation of q and k by their positions, and the write of k and v into the paged
 * cache, in one kernel.
 *   Rotation: the first rot_dim dimensions of a head are rot_dim / 2 pairs; pair j
 *   is (j, j + rot_dim / 2), or (2 j, 2 j + 1) with interleaved != 0. With
 *   p = positions[axis * ld_positions + t], axis = pair_axis[j] (pair_axis NULL: 0),
 *   c = cos_sin[p][j] and s = cos_sin[p][rot_dim / 2 + j], the pair (a, b) of
 *   token t becomes
 *     RN(RN(a c) - RN(b s)), RN(RN(b c) + RN(a s))     (binary32 roundings).
 *   Dimensions from rot_dim on stay as they are, and so does a pair whose axis
 *   is outside [0, num_axes) or whose position is outside [0, max_position).
 *   q_out = the rotated q, rounded to BF16. q NULL: heads, ld_q, q_out are not
 *   used, and k and v are written alone.
 *   Cache: row slots[t] of k_packed, k_scales gets the rotated k (its binary32
 *   values) and that of v_packed, v_scales gets v, quantized as
 *   nvfp4_quantize_paged does with k_gs and v_gs (NULL: 1.0). A token whose slot
 *   is outside [0, num_slots) is not written to the cache; its row of q_out is.
 *   Two tokens must not share a slot: the row would hold a mix of both. q_out
 *   over q, k or v, and the two caches over each other, are refused.
 * q [tokens][ld_q] BF16, heads * head_dim columns used; k, v [tokens][ld_k],
 * [tokens][ld_v], kv_heads * head_dim columns; positions num_axes rows of int32
 * [tokens]; cos_sin [max_position][rot_dim] FP32; slots [tokens] int64;
 * q_out [tokens][ld_out]; caches [num_slots][kv_heads * head_dim / 2] and
 * [num_slots][kv_heads * head_dim / 16].
 * head_dim is a multiple of 16 up to 512, rot_dim even, 0 to head_dim, num_axes 1 to 16,
 * heads and kv_heads at most 1024, tokens < 2^31, max_position < 2^31; ld_q, ld_k, ld_v,
 * ld_out multiples of 8; q, k, v, q_out, cos_sin 16-byte aligned, packed caches
 * and slots 8-byte, scale caches any. Values must be finite. tokens == 0 is a no-op.
 */
nvfp4_status_t nvfp4_rope_append(const uint16_t *q, int64_t tokens, int64_t ld_q, int32_t heads,
                                 const uint16_t *k, int64_t ld_k, const uint16_t *v, int64_t ld_v,
                                 int32_t kv_heads, int32_t head_dim, const int32_t *positions,
                                 int64_t ld_positions, int32_t num_axes, const int32_t *pair_axis,
                                 const float *cos_sin, int64_t max_position, int32_t rot_dim,
                                 int32_t interleaved, const float *k_gs, const float *v_gs,
                                 const int64_t *slots, int64_t num_slots, uint8_t *k_packed,
                                 uint8_t *k_scales, uint8_t *v_packed, uint8_t *v_scales,
                                 uint16_t *q_out, int64_t ld_out, hipStream_t stream);

/*
 * Keys of the pages that the new tokens complete: of request b the pages
 * floor((L - n) / page_size) up to floor(L / page_size) - 1 (with n = L, all its
 * complete pages). Of a page and key/value head, with the cache's values k_t
 * (E2M1 code times E4M3 scale, without the global scale),
 *   S_d = sum over the page's tokens of 2^10 k_t[d]        (a whole number),
 *   e   = max(0, bits - 7), bits the length of max_d |S_d| in binary,
 *   keys[page][head][d] = S_d / 2^e to the nearest whole number, at most 127 in
 *   magnitude; a sum half way between two goes to either (the one nearer 0 where
 *   binary64's pow(2, -e) is an ulp low, else the even one),
 *   exponents[page][head] = e.
 * page is the page's number in the cache. Other pages' keys keep their values;
 * hidden pages have none.
 * keys [num_slots / page_size][kv_heads][head_dim] int8, exponents
 * [num_slots / page_size][kv_heads] int8. max_query_len: the largest n that the
 * caller expects; it chooses the grid, not the result. head_dim is 64, 128 or
 * 256, kv_heads at most 1024, num_seqs <= 65535, num_slots < 2^31, max_pages *
 * page_size <= 2^30; k_packed 8-byte aligned, keys 16-byte. One kernel.
 */
nvfp4_status_t nvfp4_page_keys(const uint8_t *k_packed, const uint8_t *k_scales,
                               int64_t num_slots, int32_t kv_heads, int32_t head_dim,
                               int32_t page_size, const int32_t *block_table, int64_t ld_table,
                               int64_t max_pages, const int32_t *seq_lens,
                               const int32_t *query_offsets, int64_t num_seqs,
                               int64_t max_query_len, int8_t *keys, int8_t *exponents,
                               hipStream_t stream);

/*
 * The pages that each token attends to, for each key/value head. For the token at
 * position p, c = floor(p / page_size) is its own page. Listed are
 *   the pages j < first and the pages c - local < j (j <= c both), and of the
 *   others in front of c the top_k with the largest score, ties to the lower page;
 *   hidden pages are not chosen by score.
 * The score compares 8-bit queries with the page keys: with g = heads / kv_heads,
 * the head's g rows of q share
 *   e = floor(log2(max |q|)) - 6, q8 = min(127, |rint(q / 2^e)|) with q's sign,
 *   score_j = max over the rows of (sum_d q8[d] keys[page][head][d]) * 2^exponents[page][head],
 * which is exact in FP32. So keys of the pages in front of the tokens' own ones must
 * be there (nvfp4_page_keys of this and earlier steps). The global scale of the
 * keys is taken to be positive: it does not change the order.
 * pages [tokens][kv_heads][first + top_k + local] int32 gets the listed pages
 * (their place in the request, not in the cache) in ascending order, -1 behind
 * them; all -1 where p < 0. Rows of no request keep their values.
 * q must be finite (what a token with other values chooses by score is not
 * specified; its list is valid). head_dim is 64, 128 or 256; heads a multiple of
 * kv_heads, at most 1024; top_k, first >= 0, local >= 1, first + top_k + local <=
 * 2048; max_pages <= 32768 and max_pages * page_size <= 2^30; num_seqs <= 65535,
 * num_slots < 2^31, tokens * heads <= 2^23; exponents are taken to be 0 to 64; ld_q a
 * multiple of 8; q and keys 16-byte aligned. workspace:
 * nvfp4_select_pages_workspace(...) bytes (may be 0, then workspace may be NULL),
 * 16-byte aligned. One kernel, or two for few tokens.
 * max_pages is taken for the longest request's pages: it chooses the workspace and
 * the cut of the work, not the result. Of a table with more columns only those that
 * the longest request needs should be named (ld_table may be larger): 2048 tokens
 * of up to 500 pages take four times as long with 2049 columns as with 501.
 */
nvfp4_status_t nvfp4_select_pages(const uint16_t *q, int64_t tokens, int64_t ld_q, int32_t heads,
                                  int32_t kv_heads, int32_t head_dim, const int8_t *keys,
                                  const int8_t *exponents, int64_t num_slots, int32_t page_size,
                                  const int32_t *block_table, int64_t ld_table,
                                  int64_t max_pages, const int32_t *seq_lens,
                                  const int32_t *query_offsets, int64_t num_seqs, int32_t top_k,
                                  int32_t first, int32_t local, int32_t *pages, void *workspace,
                                  int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that nvfp4_select_pages needs for these sizes (the same
 * arguments as the call's), or -1 where the call refuses them. Needs no GPU. */
int64_t nvfp4_select_pages_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                     int64_t num_seqs, int64_t max_pages);

/*
 * Attention of each token over the tokens of its listed pages, as
 * nvfp4_paged_attention computes it over all of them: the token at position p,
 * query head h of it with key/value head h / (heads / kv_heads), sees the tokens
 * t <= p of the pages pages[token][kv head][i], i < list_len. Entries may stand in
 * any order; one outside [0, max_pages), a hidden page and a page behind the
 * token's own show nothing; a page listed twice counts twice. out and lse are those
 * of nvfp4_paged_attention, as are the types, layouts, roundings and limits; a row
 * that sees no token gets out = 0 and lse = -inf, rows of no request keep their
 * values. list_len is 0 to 2048, list_len * page_size <= 2^30, tokens * heads <=
 * 2^23.
 * workspace: nvfp4_sparse_attention_workspace(...) bytes (may be 0, then
 * workspace may be NULL), 16-byte aligned. One kernel, or two where a row's list
 * is split over workgroups.
 */
nvfp4_status_t nvfp4_sparse_attention(const uint16_t *q, int64_t tokens, int64_t ld_q,
                                      int32_t heads, int32_t kv_heads, int32_t head_dim,
                                      const uint8_t *k_packed, const uint8_t *k_scales,
                                      const uint8_t *v_packed, const uint8_t *v_scales,
                                      int64_t num_slots, int32_t page_size,
                                      const int32_t *block_table, int64_t ld_table,
                                      int64_t max_pages, const int32_t *seq_lens,
                                      const int32_t *query_offsets, int64_t num_seqs,
                                      const int32_t *pages, int64_t list_len, float scale,
                                      const float *k_gs, const float *v_gs, uint16_t *out,
                                      int64_t ld_out, float *lse, void *workspace,
                                      int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that nvfp4_sparse_attention needs for these sizes (the same
 * arguments as the call's), or -1 where the call refuses them. Needs no GPU. */
int64_t nvfp4_sparse_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads,
                                         int32_t head_dim, int32_t page_size,
                                         int64_t num_seqs, int64_t list_len);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_SPARSE_H */
