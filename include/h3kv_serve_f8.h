/*
 * h3kv_serve_f8.h -- C ABI of libh3kv's serving operators around two things:
 * the rotation of queries and keys by their positions, on the way into the
 * pages of h3kv_serve.h or into those declared here, and a cache in pages of
 * e4m3 codes with one scale for each page and head, with the attention that
 * reads it.
 *
 * A caller that loads the library looks these entry points up by name; the
 * conventions of h3kv_serve.h hold (strided bf16 rows, index arrays in device
 * memory that the kernels check, packed tensors, H3KV_OK for empty work).
 */
#ifndef H3KV_SERVE_F8_H
#define H3KV_SERVE_F8_H

#include "h3kv_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Angles by position: row t of `table` (fp32 [rows, dim], 16-byte aligned)
 * holds dim / 2 cosines, then dim / 2 sines.  dim: 16 .. 128, a multiple of
 * 16; the channels from dim on are not rotated.  Pair j is the channels j and
 * j + dim / 2, or (interleaved) 2 j and 2 j + 1:
 *   (a, b) -> (a cos_j - b sin_j, b cos_j + a sin_j).
 * A position out of range is reported as the index arrays' entries are, and
 * row 0 taken in its place. */
typedef struct {
  const float *table;
  int64_t rows;
  int32_t dim;
  int32_t interleaved;
} h3kv_rotation;

/* h3kv_paged_append with the rotation on the way: row i of Q and of K is
 * rotated by positions[i].  The rotated Q is rounded to bf16 and written to
 * Q_out; the rotated K is not rounded before it is quantised, and where K_out
 * is not NULL also written there in bf16 (a prompt attends to it).  Q_out may be
 * Q itself and K_out K itself (the same address and strides); otherwise no
 * output shares an element with another tensor of the call.  q_heads 0: no Q.
 * A negative rows[i] leaves the row out of the cache; its Q_out and K_out are
 * written all the same. */
h3kv_status h3kv_paged_append_rotated(const h3kv_rows *Q, int32_t q_heads, const h3kv_rows *Q_out,
                                      const h3kv_rows *K, const h3kv_rows *V, const h3kv_rows *K_out,
                                      const h3kv_rotation *rotation, const int32_t *positions, const int32_t *rows,
                                      int64_t n, const h3kv_paged_store *store, void *stream);

/* A cache of e4m3 codes in pages of page_size tokens (16, 32, 64 or 128), one
 * scale for each page and head of K and of V: a cached value is code *
 * fp16(scale).  h3kv_paged_append_f8 writes scales that are powers of two from
 * 2^-15 to 2^7, with which every value is an fp16 number; with others (positive
 * ones) it is rounded to fp16 where an operation takes 16-bit operands. */
typedef struct {
  uint8_t *k_codes; /* e4m3 [pages, kv_heads, page_size, 128] */
  uint8_t *v_codes;
  float *k_scales;  /* fp32 [pages, kv_heads] */
  float *v_scales;
  int32_t pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim; /* must be 128 */
} h3kv_paged_store_f8;

/* Bytes of the four buffers together (0 for invalid arguments, and for a store that
 * the calls refuse: more than 65535 heads, or pages * kv_heads * page_size above
 * 2^31 - 256). */
size_t h3kv_paged_store_f8_bytes(int32_t pages, int32_t kv_heads, int32_t page_size, int32_t head_dim);

/* Append the rows cu_new[i] .. cu_new[i+1]-1 of K and V (bf16 [kv_heads, n, 128])
 * as the last tokens of sequence i, which has lengths[i] tokens with them;
 * page_table: [seqs, max_pages], entry p of a sequence holding its tokens
 * p * page_size and on.  The pages written belong to that sequence alone.
 * With a rotation (NULL: none) K is rotated by positions[r] of its row r, or
 * (positions NULL) by its token's place in the sequence; Q, Q_out and K_out as
 * in h3kv_paged_append_rotated (they need a rotation).
 *
 * A page's scale is the least 2^e, -15 <= e <= 7, with which 448 * 2^e reaches
 * the size of every value the page was given since its first token was written;
 * codes are round-to-nearest-even of value / 2^e for the exactly rotated value
 * (products and sum to 2^-45 of them).  When new tokens make the scale of a
 * partly filled page grow, the codes it held are rounded anew, code * old /
 * new; a page whose first token is among the new ones starts afresh, whatever
 * it held.  A shortened sequence's last page keeps the scale it had.  Values
 * beyond 448 * 2^7 and infinities are held as that, NaN as NaN.  A tensor's rows
 * of no sequence are not read, and nothing is written for them.  (Where cu_new
 * falls, which is reported, new tokens of other sequences may be left out.)  A call may
 * mix single tokens with long chunks: it takes the time of the tokens of one to four
 * pages, one after the other, beyond that of the bytes. */
h3kv_status h3kv_paged_append_f8(const h3kv_rows *Q, int32_t q_heads, const h3kv_rows *Q_out, const h3kv_rows *K,
                                 const h3kv_rows *V, const h3kv_rows *K_out, const h3kv_rotation *rotation,
                                 const int32_t *positions, int64_t n, const h3kv_paged_store_f8 *store,
                                 const int32_t *page_table, int64_t max_pages, const int32_t *lengths,
                                 const int32_t *cu_new, int32_t seqs, void *stream);

/* h3kv_paged_read of these pages: the values in fp16, rounded to bf16. */
h3kv_status h3kv_paged_read_f8(const h3kv_paged_store_f8 *store, const int32_t *rows, int64_t n, const h3kv_rows *K,
                               const h3kv_rows *V, void *stream);

/* h3kv_paged_copy of these pages; n is at most 2^27 - 16, and less where a page's
 * codes of all heads take more than 128 KB: n * 2 * (16 KB pieces of them) < 2^31. */
h3kv_status h3kv_paged_copy_f8(const h3kv_paged_store_f8 *store, const int32_t *src, const int32_t *dst, int64_t n,
                               void *stream);

/* Most rows of Q in one call of h3kv_attend_paged_f8. */
#define H3KV_PAGED_MAX_ROWS (1 << 20)

/* Device bytes of h3kv_attend_paged_f8's workspace (0 for invalid arguments),
 * used as that of h3kv_attend_tree. */
size_t h3kv_attend_paged_f8_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t n, int32_t seqs);

/* Causal attention of each sequence's last tokens over its cache, with grouped
 * heads: rows cu_q[i] .. cu_q[i+1]-1 of Q are the last m of the lengths[i]
 * tokens of sequence i (appended before), one or many of them, and the last
 * row sees every token, each row before it one less.
 *   S = Q K'^T softmax_scale, O = bf16(softmax(S) V'), K' and V' the cached
 *   values; weights rounded to fp16 for the second product (down to 2^-32 of the
 *   largest), fp32 sums;  softmax_scale and lse as h3kv_attend_tree.
 * A query row is taken times a power of two.  For few rows as fp16, exact for
 * elements down to 2^-32 of the row's largest and within 2^-40 of that below; for
 * many as the sum of two e4m3 parts, exact down to 2^-9 of the largest and within
 * 2^-17 of that below, or within 2^-76 (a row with channels far above the rest keeps
 * fewer bits of these).  A row of Q with an element beyond 65504, an infinity or NaN
 * gives an undefined row of O.
 * A cached row that is not finite may reach every row of its own
 * sequence, and none of another's.  Splitting of the keys, determinism and the
 * workspace are those of h3kv_attend_tree.  The kernel is chosen by the mean
 * count of rows, q_heads n / (kv_heads seqs) -- up to 16 for few, from 33 on for
 * many, between them by the tokens that max_pages can hold -- so a call that mixes
 * single tokens with long chunks is right, but slower than one call for each (1.4 to
 * 2 times where measured). */
h3kv_status h3kv_attend_paged_f8(const h3kv_rows *Q, int32_t q_heads, int64_t n, const h3kv_paged_store_f8 *store,
                                 const int32_t *page_table, int64_t max_pages, const int32_t *lengths,
                                 const int32_t *cu_q, int32_t seqs, float softmax_scale, const h3kv_rows *O,
                                 float *lse, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* H3KV_SERVE_F8_H */
