/*
 * kv8.h -- INT8 key/value cache with one scale per page of tokens and head, and
 * attention over it, on AMD Instinct MI355X (gfx950). Part of libw4a4.so; the
 * conventions of w4a4.h hold (device pointers, validation first, asynchronous
 * on `stream`, no allocation, status codes).
 *
 * The pool. `num_pages` pages, each holding `page` consecutive positions of one
 * sequence for `heads` kv heads of `dim` dimensions:
 *   k_cache  int8 [num_pages][heads][page][dim]
 *   v_cache  int8 [num_pages][heads][dim][page]   (positions contiguous)
 *   k_scale, v_scale  f32 [num_pages][heads]
 * A key is k_scale * code, a value v_scale * code.
 *   page: 16, 32, 64, 128 or 256; dim: 64, 128, 192 or 256; caches 16-byte
 *   aligned, scales 4-byte aligned; heads <= 16384.
 *
 * The batch. B sequences packed along T tokens:
 *   block_table  int32 [B][table_ld]: the page of positions page * j ..
 *                page * j + page - 1 of sequence b is block_table[b][j]
 *   cu_seqlens   int32 [B + 1], not decreasing: tokens cu_seqlens[b] ..
 *                cu_seqlens[b + 1] - 1 of the packed tensors are the new tokens
 *                of sequence b
 *   seq_lens     int32 [B]: its positions in the cache, the new tokens included:
 *                its n new tokens are positions seq_lens[b] - n .. seq_lens[b] - 1
 *   max_new      at least every sequence's number of new tokens
 *   max_len      at least every seq_lens[b], at most table_ld * page
 *   B <= 65535; T and max_len < 2^28
 * These four are read on the device: nothing synchronizes, and a captured call
 * follows the values at replay. More new tokens than max_new are read as max_new,
 * a length above max_len as max_len, so that no access leaves the tensors; tokens at negative positions (n > seq_lens[b]) are not stored, read
 * as zeros and see nothing; table entries that are no page of the pool are
 * skipped (not stored, read as zeros, masked). Table entries past a sequence's
 * last position are never read. Tokens of the packed tensors that belong to no
 * sequence are left as they are.
 */
#ifndef KV8_H
#define KV8_H

#include "w4a4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Store the new tokens' keys and values. For each page and kv head that
 * receives tokens, with s_old its scale if the page already holds earlier
 * positions of the sequence and 0 otherwise (a reused page starts afresh):
 *   s = max(s_old, fl32(max|new| / 127))
 *   earlier codes, if s > s_old:  q <- rne(fl32(q * fl32(s_old / s)))
 *   new codes:                    rne(fl32(x / s))  (s = 0: 0)
 * Each growth of a page's scale rounds its older codes again, by half a step at
 * most: after g growths a value is within (g + 1) / 2 steps s of what was stored (its
 * steps never shrink), so a page whose maximum rises with every token may be off by
 * page / 2 steps at its first tokens; one whose largest values come first, by 1/2.
 * Other slots keep their bytes. The pages written must not be shared. A NaN or an
 * infinity among the new values makes s NaN (the codes of the new tokens are then
 * any), until the page is used afresh.
 *
 *   k, v    new keys and values, token t of head h at k + t * k_tok + h * k_head
 *           (elements), dim contiguous; x_dtype W4A4_Y_F16 or W4A4_Y_BF16;
 *           16-byte aligned, strides multiples of 8
 */
w4a4_status_t kv8_append(const void* k, const void* v, int32_t x_dtype, int64_t k_tok, int64_t k_head,
                         int64_t v_tok, int64_t v_head,
                         int8_t* k_cache, int8_t* v_cache, float* k_scale, float* v_scale,
                         int64_t num_pages, int32_t heads, int32_t page, int32_t dim,
                         const int32_t* block_table, int64_t table_ld, const int32_t* cu_seqlens,
                         const int32_t* seq_lens, int64_t B, int64_t T, int64_t max_new, int64_t max_len,
                         void* stream);

/*
 * Read cached tokens back as values (the last n positions of each sequence,
 * n from cu_seqlens as for kv8_append, whose mirror this is).
 *   k, v    out: [T][heads][dim] of y_dtype (any), aligned to 16 bytes
 */
w4a4_status_t kv8_gather(const int8_t* k_cache, const int8_t* v_cache, const float* k_scale, const float* v_scale,
                         int64_t num_pages, int32_t heads, int32_t page, int32_t dim,
                         const int32_t* block_table, int64_t table_ld, const int32_t* cu_seqlens,
                         const int32_t* seq_lens, int64_t B, int64_t T, int64_t max_new, int64_t max_len,
                         void* k, void* v, int32_t y_dtype, void* stream);

/*
 * Attention of the new tokens' queries over the cache (the new tokens already
 * stored). A query at position p sees positions j < seq_lens[b], with `causal`
 * also j <= p, with window > 0 also j > p - window:
 *   o = sum_j softmax_j(scale * q . k_j) v_j;  lse = ln sum_j exp(scale * q . k_j)
 * and o = 0, lse = -inf where it sees none. Query head h reads kv head
 * h / (q_heads / heads).
 *
 * One kernel, chosen by max_new, serves all sequences of a call. Sequences with a
 * single new token run several times faster in a call of their own than beside long
 * chunks: put them first or last, and give each call its part of block_table,
 * cu_seqlens (which need not start at 0) and seq_lens. Rows of y that belong to no
 * sequence are left alone, so both may fill one y.
 *
 *   q       [T][q_heads] rows of dim elements at strides q_tok, q_head
 *           (elements, multiples of 8), 16-byte aligned, x_dtype W4A4_Y_F16 or
 *           W4A4_Y_BF16; q_heads a multiple of heads
 *   y       out: [T][q_heads][dim] of y_dtype (any)
 *   lse     out: f32 [T][q_heads], or NULL
 *   workspace  device memory of at least kv8_attention_workspace(...) bytes,
 *           16-byte aligned, overwritten; may be NULL when that size is 0
 * Codes enter the matrix products exactly; softmax statistics and sums are
 * fp32. A weight (softmax numerator times its page's value scale) is rounded to
 * 11 bits, or, where it is under 2^-29 of the largest such, to 2^-40 of the
 * largest page scale (2^-120, where all are smaller); with more than 128 query
 * rows per kv head (64, where the short contexts of 256 and more pairs of sequence
 * and kv head fill the GPU, or dim > 128) 2^-23 and 2^-34; bf16 queries lose elements
 * under 2^-39 of a row's largest. Scales are finite and >= 0; scores may take any
 * size that fp32 holds. A page whose key or value scale is NaN gives NaN to every
 * query that sees one of its positions, and may to others of its sequence.
 * Results do not depend on the order in which workgroups run.
 */
w4a4_status_t kv8_attention(const void* q, int32_t x_dtype, int64_t q_tok, int64_t q_head, int32_t q_heads,
                            const int8_t* k_cache, const int8_t* v_cache, const float* k_scale, const float* v_scale,
                            int64_t num_pages, int32_t heads, int32_t page, int32_t dim,
                            const int32_t* block_table, int64_t table_ld, const int32_t* cu_seqlens,
                            const int32_t* seq_lens, int64_t B, int64_t T, int64_t max_new, int64_t max_len,
                            float scale, int32_t causal, int64_t window, void* workspace, int64_t workspace_bytes,
                            void* y, int32_t y_dtype, float* lse, void* stream);

/* Workspace bytes kv8_attention needs, or -1 for invalid arguments. Host-only. */
int64_t kv8_attention_workspace(int32_t q_heads, int32_t heads, int32_t page, int32_t dim, int64_t B, int64_t T,
                                int64_t max_new, int64_t max_len, int32_t causal, int64_t window);

#ifdef __cplusplus
}
#endif

#endif /* KV8_H */
