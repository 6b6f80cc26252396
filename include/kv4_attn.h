/*
 * kv4_attn.h -- C ABI of the decode step's attention block (libmoe_tail.so): what makes the
 * attention output that moe_tail_run_attn (moe_tail.h) projects and feeds to the layer tail.
 *
 *   moe_step_tables    block tables, row starts, positions and cache slots of a step, built on
 *                      the GPU from the requests' lengths
 *   moe_qk_norm_rope   RMSNorm of every query and key head and the position rotation
 *   moe_kv4_append     keys and values of the step's rows into a paged 4-bit cache
 *   moe_kv4_read       rows of that cache back as bf16
 *   moe_kv4_attention  attention of the step's query rows over the cache
 *
 * All are stateless: borrowed device pointers, nothing allocated, no synchronisation, valid in
 * CUDA graph capture; a call runs on the current device, which must be the one that `stream`
 * and the pointers belong to.  Calls in different streams are independent as long as they share
 * no output (and no workspace).  Return codes are those of moe_tail.h (moe_tail_strerror and
 * moe_tail_last_cuda_error apply); a refused call launches nothing.
 *
 * What only the device can see (lengths, slots, page numbers) is checked on the device: the
 * kernels never leave the given buffers, and what they skip or find is reported as bits that are
 * OR-ed into *status, an int32 in device memory (NULL: not reported; the caller zeroes it).
 *
 * Cache format.  uint8 [n_pages][kv_heads][page_size / 16][17 * D]: a page holds page_size
 * consecutive tokens of one request (a multiple of 16), slot = page * page_size + offset.  Keys
 * and values are OCP MXFP4, as the layer tail's expert weights: E2M1 codes and one E8M0 scale
 * 2^(s-127) for each 32 channels of a token and head, the smallest power of two from 2^-126 to
 * 2^125 with max |x| <= 6 * 2^(s-127), codes rounded to nearest, ties to even (magnitudes past
 * 6 * 2^125 saturate there: the next code would stand for 2^128); a block of 32 with an infinity
 * or a NaN gets the scale byte 255, which stands for NaN (its codes are 0).  The scale byte 0 is
 * read as 0 (nothing writes it but the caller's memset: a zeroed cache holds zeros); 253 and 254
 * are not part of the format.
 * One tile of 16 tokens (t = 0..15, channel d = 0..D-1) of one head is 17 * D bytes: 8 D bytes of
 * key codes, 8 D of value codes, D/2 key scale bytes, D/2 value scale bytes, each in the order in
 * which the lanes (g, c), g = 0..7, c = 0..3, of the matrix instructions read them:
 *   key code of (t, d):   lane (t % 8, d % 32 / 8); byte n = t/8 * D/8 + d/32 * 4 + d%8 / 2 of it
 *   value code of (t, d): lane (d % 32 / 4, t % 8 / 2);
 *                         byte n = (t/8 * 2 + t%2) * D/16 + d/32 * 2 + d%4 / 2 of it
 *     where byte n of lane (g, c) stands at n/16 * 512 + (4 g + c) * 16 + n % 16, and even
 *     channels are its low four bits;
 *   key scale of (t, block b = d/32):   byte t%8 * D/16 + t/8 * D/32 + b
 *   value scale of (t, b):              byte t%8/2 * D/8 + 4 b + t/8 * 2 + t%2
 */
#ifndef KV4_ATTN_H
#define KV4_ATTN_H

#include "moe_tail.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of a *status word.  MOE_TAIL_STATUS_TIMEOUT may join them: a hand-over inside the attention did
 * not come in some 0.1 s, and the rows that were to come of it are NaN. */
#define MOE_KV4_STATUS_BAD_LENGTH 16 /* a negative length, one past its table row, row starts
                                        that descend or pass the call's rows; the request is
                                        skipped (its cache length cut to its table row by the
                                        attention) */
#define MOE_KV4_STATUS_NO_PAGES 32   /* the free pages ran out: table entries and slots are -1 */
#define MOE_KV4_STATUS_ROWS 64       /* the step has more rows than max_rows: it was cut to these */
#define MOE_KV4_STATUS_BAD_SLOT 128  /* a slot past the cache: the row was skipped */
#define MOE_KV4_STATUS_BAD_PAGE 256  /* a page number outside the cache: its tokens are masked */

/* Limits. */
#define MOE_KV4_MAX_REQS 1024
#define MOE_KV4_MAX_PAGE 1024

/* Tables of one step, from lengths: request r has cached_lens[r] tokens in the cache and
 * new_lens[r] rows in this step (0: none).  Where all rows are more than max_rows (status ROWS),
 * the step is cut to its first max_rows: new[r] below is what is left of new_lens[r], so that the
 * tables are those of a step with these fewer rows, and the caller may send the others in the next.
 *   row_starts[r]  = sum of new[0 .. r-1], row_starts[reqs] = all rows T
 *   kv_lens[r]     = cached_lens[r] + new[r]
 *   row i of request r (row_starts[r] <= i < row_starts[r+1]):
 *     positions[i] = cached_lens[r] + i - row_starts[r]
 *     slots[i]     = block_table[r][positions[i] / page_size] * page_size
 *                    + positions[i] % page_size
 *   rows T .. max_rows-1 (a padded step): position 0, slot -1 (moe_kv4_append skips them)
 *   block_table[r] holds the pages of the cached tokens, ceil(cached / page_size) entries; the
 *   entries up to ceil(kv_len / page_size) are filled with the next pages of free_pages, in
 *   request order; the others stay as they were
 *   *pages_used    = number of free pages taken
 * An invalid request (status BAD_LENGTH) has no rows, takes no pages and gets kv_len 0.
 * reqs 1..1024, max_rows 1..2^24, page_size a multiple of 16 up to 1024, n_free >= 0,
 * table_width >= 1 entries per request, table_stride >= table_width (entries between rows).
 * int32 arrays, slots int64; free_pages may be NULL when n_free is 0.  The outputs must not
 * overlap the inputs or one another. */
int moe_step_tables(int32_t reqs, int32_t max_rows, int32_t page_size, int32_t n_free,
                    int32_t table_width, int64_t table_stride, const int32_t* cached_lens,
                    const int32_t* new_lens, const int32_t* free_pages, int32_t* block_table,
                    int32_t* row_starts, int32_t* kv_lens, int32_t* positions, int64_t* slots,
                    int32_t* pages_used, int32_t* status, void* stream);

/* For each row t and head (q heads with q_gamma, k heads with k_gamma):
 *   n = x / sqrt(mean(x^2) + eps) * gamma
 *   for i < rot_dim / 2, a = positions[t] * inv_freq[i]: the pair
 *     (n[i], n[i + rot_dim/2]), or with `interleaved` (n[2i], n[2i+1]),
 *   turns by a: (x, y) -> (x cos a - y sin a, y cos a + x sin a); channels from rot_dim on stay
 *   out = bf16 of that (one rounding)
 *   q [rows, q_heads, D], k [rows, k_heads, D] bf16: a row's heads are contiguous, rows are
 *   ld_q, ld_k elements apart (a slice of a packed projection); q_out, k_out likewise with
 *   ld_qo, ld_ko; q_out may be q and k_out k (with equal strides), otherwise no overlap
 *   q_gamma, k_gamma bf16 [D]; NULL: that side is not normalised, only rotated (as with gamma 1
 *   and 1 / sqrt(..) left out)
 *   positions int32 [rows] (any value), inv_freq float [rot_dim / 2]; the angle is formed and
 *   reduced in 64 bits, so far positions keep full precision
 * rows 1..2^24, q_heads 1..1024, k_heads 0..1024 (0: k, k_out, k_gamma may be NULL), D a multiple
 * of 16 in [16, 256], rot_dim a multiple of 16 in [0, D], eps > 0; tensors 16-byte aligned, row
 * strides multiples of 8 (at least heads * D). */
int moe_qk_norm_rope(int32_t rows, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                     int32_t rot_dim, int32_t interleaved, float eps, const void* q, int64_t ld_q,
                     const void* k, int64_t ld_k, const void* q_gamma, const void* k_gamma,
                     const int32_t* positions, const float* inv_freq, void* q_out, int64_t ld_qo,
                     void* k_out, int64_t ld_ko, void* stream);

/* Quantise the rows' keys and values into their slots of the cache.
 *   k, v bf16 [rows, kv_heads, D], row strides ld_k, ld_v in elements
 *   slots int64 [rows]; negative: the row is skipped; the slots of one call are distinct (of two
 *   rows with the same slot the cache holds a mixture; no other slot is touched)
 * rows 1..2^24, kv_heads 1..256, D in {64, 128, 256}, page_size a multiple of 16 up to 1024,
 * n_pages 1..2^31-1; k, v and cache 16-byte aligned, strides multiples of 8 (at least
 * kv_heads * D). */
int moe_kv4_append(int32_t rows, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                   int64_t n_pages, void* cache, const void* k, int64_t ld_k, const void* v,
                   int64_t ld_v, const int64_t* slots, int32_t* status, void* stream);

/* The values that the cache holds in the given slots, as bf16 (exact): the inverse of
 * moe_kv4_append; rows with a negative slot or one past the cache are left as they were.  Same
 * arguments; a slot may come up more than once. */
int moe_kv4_read(int32_t rows, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                 int64_t n_pages, const void* cache, void* k, int64_t ld_k, void* v, int64_t ld_v,
                 const int64_t* slots, int32_t* status, void* stream);

/* Attention over the cache.  Request r has the query rows row_starts[r] .. row_starts[r+1]-1,
 * the last of its kv_lens[r] cache tokens: row i stands at position
 *   p = kv_lens[r] - (row_starts[r+1] - i)
 * and sees the tokens j <= p with window == 0, or j > p - window, or j < sinks.  Query head h
 * reads kv head h / (q_heads / kv_heads):
 *   out[i][h] = bf16( sum_j softmax_j(scale * q[i][h] . K[j]) V[j] ),   0 if it sees none
 *   q bf16 [rows, q_heads, D], out likewise, row strides ld_q, ld_o in elements; out must not
 *   overlap an input
 *   block_table int32 [reqs] rows of table_width entries, table_stride apart
 * Rows that no request has (from row_starts[reqs] on) are left as they were; a row that two requests
 * have, which takes row starts that descend between them (BAD_LENGTH), holds what either gives it.  `max_new` is the
 * caller's estimate of the largest number of rows of a request; it steers how the work is cut
 * and does not change what is computed.  `workspace` (16-byte aligned, exclusive to the call
 * until it has completed) holds workspace_bytes >= moe_kv4_attention_workspace(..) with the same
 * arguments on this device.
 * Arithmetic: queries and cached keys enter the scores exactly (tf32 holds both), scores, scale,
 * softmax statistics and output sums are fp32; the softmax numerators are rounded to tf32 for the
 * product with the exact values, the sum that divides takes them unrounded.  A numerator may reach
 * 2^40 (the reference is not always the maximum), so sums of values past 2^60 or so may overflow.
 * The split of the work depends on the lengths of all requests and on the device, so the same
 * request in another batch may differ in the last bits; the same call always gives the same bits.
 * rows 1..2^20, reqs 1..1024, kv_heads 1..256, q_heads a multiple of it with q_heads / kv_heads
 * <= 256, D in {64, 128, 256}, page_size a multiple of 16 up to 1024, n_pages 1..2^31-1,
 * scale finite and > 0, window >= 0, sinks >= 0 (ignored when window == 0), max_new >= 1; q, out,
 * cache 16-byte aligned, strides multiples of 8 (at least q_heads * D).  A call whose requests
 * would read more than 2^31 - 1 tiles (of 16 tokens, once for each kv head and up to 32 rows, and
 * 36 more for each of those) sets BAD_LENGTH and computes nothing: its rows are NaN. */
int moe_kv4_attention(int32_t rows, int32_t reqs, int32_t q_heads, int32_t kv_heads,
                      int32_t head_dim, int32_t page_size, int64_t n_pages, const void* q,
                      int64_t ld_q, const void* cache, const int32_t* block_table,
                      int32_t table_width, int64_t table_stride, const int32_t* row_starts,
                      const int32_t* kv_lens, float scale, int32_t window, int32_t sinks,
                      int32_t max_new, void* out, int64_t ld_o, void* workspace,
                      size_t workspace_bytes, int32_t* status, void* stream);

/* Bytes of workspace for moe_kv4_attention on the current device; negative on error
 * (MOE_TAIL_ERR_UNSUPPORTED for a shape it does not take, MOE_TAIL_ERR_CUDA without a device). */
int64_t moe_kv4_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                    int32_t max_new);

#ifdef __cplusplus
}
#endif

#endif /* KV4_ATTN_H */
