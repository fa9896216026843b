/*
 * h3kv_serve.h -- C ABI of libh3kv's serving operators: causal attention over
 * packed prompts with grouped heads, and a kvi8r cache in pages that grows
 * token by token -- rows written and read, pages copied, drafted rows kept or
 * dropped -- with the attention of a tree of drafted tokens (a single new
 * token is the tree of one node) over it.
 *
 * ABI version 9 libraries exist without these entry points: a caller that loads
 * the library looks them up by name.
 *
 * The conventions of h3kv.h hold here too: host-side checks before any
 * launch, stream-ordered asynchronous calls, memory owned by the caller,
 * bounded waits.  What differs:
 *  - bf16 tensors [heads, rows, 128] may be strided (h3kv_rows), since the
 *    projections before them leave the heads of a token side by side.
 *  - Index arrays (row and page numbers, lengths, cumulative counts, parents)
 *    are int32 in device memory, so that a captured graph takes new ones at
 *    each replay.  The host cannot check them: a kernel that meets an entry
 *    out of range leaves that entry's work out, touches no memory that it
 *    names (h3kv_attend_tree reads page 0 in the place of such a page), and
 *    h3kv_sync_status() then returns H3KV_ERR_DEVICE_DATA.  The output of the
 *    sequence concerned is undefined.
 *  - Packed tensors: the rows cu[i] .. cu[i+1]-1 belong to sequence i.  Rows
 *    before cu[0] and from cu[seqs] on belong to none; nothing is written for
 *    them.
 *  - What a call writes shares no memory with what else it reads or writes:
 *    H3KV_ERR_INVALID_ARG, by the tensors' extents.  K and V of a read may take
 *    turns in one buffer (equal strides), and O of the attention calls may lie
 *    beside Q, K and V in one; O is not compared with those.
 *  - H3KV_OK for empty work (no rows, no sequences), with nothing launched.
 */
#ifndef H3KV_SERVE_H
#define H3KV_SERVE_H

#include "h3kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bf16 [heads, rows, 128]: the 128 values of a row are contiguous, strides
 * are in elements and multiples of 8, `data` is 16-byte aligned. */
typedef struct {
  uint16_t *data;
  int64_t head_stride;
  int64_t row_stride;
} h3kv_rows;

/* A kvi8r cache in pages of page_size tokens (16, 32, 64 or 128).  Codes and
 * scales of a row have the format and the formula of h3kv_store with one scale
 * per row.  h3kv_paged_append does not compute them as h3kv_build_store does:
 * next to a rounding border a scale may differ by one fp16 step, a code by
 * one.  Row number r of the pool is slot r % page_size of page r / page_size. */
typedef struct {
  int8_t *k_codes;    /* [pages, kv_heads, page_size, 128] */
  int8_t *v_codes;
  uint16_t *k_scales; /* fp16 [pages, kv_heads, page_size] */
  uint16_t *v_scales;
  int32_t pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim;   /* must be 128 */
} h3kv_paged_store;

/* Bytes of the four buffers together, 2 pages kv_heads page_size 130 (0 for
 * invalid arguments, among them pages * page_size above 2^31 - 256). */
size_t h3kv_paged_store_bytes(int32_t pages, int32_t kv_heads, int32_t page_size, int32_t head_dim);

/* Rotate and quantise the n rows of K and V (bf16 [kv_heads, n, 128]) and
 * write row i to pool row rows[i]; a negative rows[i] leaves the row out.  No
 * pool row may be named twice in one call.  A row that holds a NaN gets a scale
 * of NaN: it reads back as NaN, and so does what attends to it. */
h3kv_status h3kv_paged_append(const h3kv_rows *K, const h3kv_rows *V, const int32_t *rows, int64_t n,
                              const h3kv_paged_store *store, void *stream);

/* Pool rows rows[0 .. n-1], dequantised (fp16(code * scale)), un-rotated and
 * rounded to bf16, into K and V [kv_heads, n, 128]; a negative rows[i] (and
 * one out of range) gives a row of zeros. */
h3kv_status h3kv_paged_read(const h3kv_paged_store *store, const int32_t *rows, int64_t n, const h3kv_rows *K,
                            const h3kv_rows *V, void *stream);

/* Copy page src[i] to page dst[i] (codes and scales of every head), i < n; a
 * pair with a negative entry is left out.  No page may be a dst twice, or
 * both a dst and a src, in one call. */
h3kv_status h3kv_paged_copy(const h3kv_paged_store *store, const int32_t *src, const int32_t *dst, int64_t n,
                            void *stream);

/* Most drafted nodes of one sequence in h3kv_paged_keep and h3kv_attend_tree. */
#define H3KV_TREE_MAX_NODES 64

/* Of each sequence's last m = cu_nodes[i+1] - cu_nodes[i] cached rows, move
 * those with keep[cu_nodes[i] + j] != 0 to the places behind the rows before
 * them, in order, and write the length that is left to new_lengths[i]
 * (another array than lengths).  The pages of those rows belong to this
 * sequence alone.  page_table: [seqs, max_pages], entry p of a sequence
 * holding its tokens p * page_size and on; keep: one byte for each node. */
h3kv_status h3kv_paged_keep(const h3kv_paged_store *store, const int32_t *page_table, int64_t max_pages,
                            const int32_t *lengths, const int32_t *cu_nodes, int32_t seqs, const uint8_t *keep,
                            int64_t nodes, int32_t *new_lengths, void *stream);

/* Device bytes of h3kv_attend_tree's workspace (0 for invalid arguments),
 * which is 32-byte aligned.  It needs no initial value; calls that overlap on the GPU (two streams, two
 * replayed graphs) must not share it. */
size_t h3kv_attend_tree_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t nodes, int32_t seqs);

/* Attention of drafted tokens over the paged cache, with grouped heads: q head
 * h reads kv head h / (q_heads / kv_heads).  Sequence i has lengths[i] cached
 * rows; the last m = cu_nodes[i+1] - cu_nodes[i] (at most 64) of them are the
 * drafted nodes themselves, appended before this call.  Node j (row
 * cu_nodes[i] + j of Q) sees every row before the drafted ones and the nodes
 * on the path from itself to its root: itself, parents[cu_nodes[i] + j], that
 * node's parent and so on.  A parent is the number of an earlier node of the
 * same sequence; any other value (-1, say) makes the node a root.  parents
 * NULL: node j's parent is j - 1, a plain run of tokens.
 *   q' = fp16(Q H), K' = fp16(code * scale), V' likewise;
 *   S = q' K'^T softmax_scale;  O = bf16((softmax(S) V') H), weights rounded to
 *   fp16 for the second product (down to 2^-32 of the largest), fp32 sums;
 *   lse = ln(sum exp S), fp32 [q_heads, nodes] contiguous, or NULL.
 * softmax_scale <= 0 selects 1/sqrt(128).  nodes: the rows of Q.
 * A cached row that is not finite (a scale of NaN, or code * scale beyond fp16)
 * may reach every node of its own sequence, also those that do not see it, and
 * none of another's.
 * q_heads / kv_heads is at most 64.  The kernel is chosen by the mean count of
 * rows, q_heads nodes / (kv_heads seqs), since the host does not know the single
 * counts: sequences without nodes among seqs make one with many slow, not
 * wrong.  The keys of a sequence are split over
 * the GPU's SMs and joined by their log-sum-exp in a fixed order: the same
 * call gives the same bits, another batch around a sequence may round
 * differently. */
h3kv_status h3kv_attend_tree(const h3kv_rows *Q, int32_t q_heads, int64_t nodes, const h3kv_paged_store *store,
                             const int32_t *page_table, int64_t max_pages, const int32_t *lengths,
                             const int32_t *cu_nodes, int32_t seqs, const int32_t *parents, float softmax_scale,
                             const h3kv_rows *O, float *lse, void *workspace, size_t workspace_bytes, void *stream);

/* Attention over packed prompts, with grouped heads as above: sequence i owns
 * the rows cu_q[i] .. cu_q[i+1]-1 of Q and O [q_heads, q_rows, 128] and the
 * rows cu_k[i] .. cu_k[i+1]-1 of K and V [kv_heads, k_rows, 128].  causal: the
 * last query row sees every key and each row before it one key less (row t of
 * nq sees the keys u <= t + nk - nq of nk), so a chunk of a prompt attends
 * behind its prefix; otherwise every row sees every key of its sequence.
 *   S = Q K^T softmax_scale; O = bf16(softmax(S) V), P rounded to bf16 for
 *   the second product, fp32 accumulation; lse as above, or NULL.
 * Scores are held in fp32 and may have any size that fp32 holds; a row with one
 * of +infinity is undefined.  A row that sees no key (or only scores of
 * -infinity) gets O = 0 and lse = -infinity.  A value of K or V that is infinite
 * or NaN reaches no row of another sequence; within its own it may reach rows
 * that do not see it (a weight of 0 times such a value of V). */
h3kv_status h3kv_attend_prompt(const h3kv_rows *Q, int32_t q_heads, int64_t q_rows, const h3kv_rows *K,
                               const h3kv_rows *V, int32_t kv_heads, int64_t k_rows, const int32_t *cu_q,
                               const int32_t *cu_k, int32_t seqs, int32_t causal, float softmax_scale,
                               const h3kv_rows *O, float *lse, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* H3KV_SERVE_H */
