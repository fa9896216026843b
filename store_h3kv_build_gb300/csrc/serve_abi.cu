// serve_abi.cu -- the C ABI of the serving operators (h3kv_serve.h): host-side
// argument checks and the launches.
#include <math.h>

#include "serve.h"
#include "spans.h"

namespace {

using h3kv::meet;
using h3kv::meets_any;
using h3kv::meets_store;
using h3kv::rows_meet;
using h3kv::Span;
using h3kv::span;

// Rows are addressed with 32-bit numbers.
constexpr int64_t kMaxRows = (1ll << 31) - 256;
constexpr int64_t kMaxStride = (1ll << 38) - 8;  // elements; a tensor map's stride is below 2^40 bytes
constexpr int32_t kMaxHeads = 65535;
constexpr int32_t kMaxGroup = 64;
constexpr int32_t kMaxSeqs = 65535;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides that a tensor map takes: no axis of more than one entry is
// broadcast (stride 0) or has rows that overlap.
bool rows_ok(const h3kv_rows *r, int64_t heads, int64_t rows) {
  return r && r->data && aligned(r->data, 16) && r->head_stride % 8 == 0 && r->row_stride % 8 == 0 &&
         (heads <= 1 || (r->head_stride >= H3KV_HEAD_DIM && r->head_stride <= kMaxStride)) &&
         (rows <= 1 || (r->row_stride >= H3KV_HEAD_DIM && r->row_stride <= kMaxStride));
}
// An output's rows do not lie over each other.
bool out_rows_ok(const h3kv_rows *r, int64_t heads, int64_t rows) {
  if (!rows_ok(r, heads, rows)) return false;
  if (heads <= 1 || rows <= 1) return true;
  const int64_t hs = r->head_stride, rs = r->row_stride;
  return hs >= rs ? hs >= (rows - 1) * rs + H3KV_HEAD_DIM : rs >= (heads - 1) * hs + H3KV_HEAD_DIM;
}

h3kv_status paged_args(const h3kv_paged_store *st, h3kv::PagedArgs *out) {
  if (!st || st->pages < 0 || st->kv_heads < 0 || st->kv_heads > kMaxHeads) return H3KV_ERR_INVALID_ARG;
  if (st->head_dim != H3KV_HEAD_DIM) return H3KV_ERR_UNSUPPORTED;
  const int32_t ps = st->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128) return H3KV_ERR_INVALID_ARG;
  // row numbers, and rows of all heads, in 31 bits
  if (static_cast<int64_t>(st->pages) * ps > kMaxRows / (st->kv_heads > 0 ? st->kv_heads : 1))
    return H3KV_ERR_INVALID_ARG;
  if (st->pages > 0 && st->kv_heads > 0) {
    if (!st->k_codes || !st->v_codes || !st->k_scales || !st->v_scales) return H3KV_ERR_INVALID_ARG;
    if (!aligned(st->k_codes, 16) || !aligned(st->v_codes, 16) || !aligned(st->k_scales, 16) ||
        !aligned(st->v_scales, 16))
      return H3KV_ERR_INVALID_ARG;
  }
  out->k_codes = st->k_codes;
  out->v_codes = st->v_codes;
  out->k_scales = st->k_scales;
  out->v_scales = st->v_scales;
  out->pages = st->pages;
  out->kv_heads = st->kv_heads;
  out->page_size = ps;
  out->page_shift = ps == 16 ? 4 : ps == 32 ? 5 : ps == 64 ? 6 : 7;
  out->err = nullptr;
  return H3KV_OK;
}

h3kv_status status_of(cudaError_t e) { return e == cudaSuccess ? H3KV_OK : H3KV_ERR_CUDA; }

float scale_log2_of(float softmax_scale) {
  const float s = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(128.0f);
  return s * 1.4426950408889634f;
}

// The limit of a wait for the end of a segment of up to `keys` keys: that of a
// wait for each key tile (where a tile hangs, its own wait runs out first and
// ends this one).
uint64_t segment_timeout(uint64_t timeout_ns, int64_t keys) {
  const uint64_t n = static_cast<uint64_t>(keys) / H3KV_KV_TILE + 8;
  return timeout_ns > UINT64_MAX / n ? UINT64_MAX : timeout_ns * n;
}

// Page tables are addressed as [seqs, max_pages] of 4-byte entries.
bool table_ok(const int32_t *page_table, int64_t max_pages) {
  return max_pages >= 0 && max_pages <= kMaxRows / 16 && aligned(page_table, 4) && (page_table || max_pages == 0);
}

}  // namespace

extern "C" {

size_t h3kv_paged_store_bytes(int32_t pages, int32_t kv_heads, int32_t page_size, int32_t head_dim) {
  if (pages < 0 || kv_heads < 0 || head_dim != H3KV_HEAD_DIM) return 0;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return 0;
  if (static_cast<int64_t>(pages) * page_size > kMaxRows) return 0;
  return static_cast<size_t>(2) * static_cast<size_t>(pages) * static_cast<size_t>(kv_heads) *
         static_cast<size_t>(page_size) * (H3KV_HEAD_DIM + 2);
}

h3kv_status h3kv_paged_append(const h3kv_rows *K, const h3kv_rows *V, const int32_t *rows, int64_t n,
                              const h3kv_paged_store *store, void *stream) {
  h3kv::PagedArgs p;
  h3kv_status st = paged_args(store, &p);
  if (st != H3KV_OK) return st;
  if (n < 0 || n > kMaxRows) return H3KV_ERR_INVALID_ARG;
  if (n == 0 || p.kv_heads == 0) return H3KV_OK;
  if (!rows_ok(K, p.kv_heads, n) || !rows_ok(V, p.kv_heads, n) || !rows || !aligned(rows, 4)) return H3KV_ERR_INVALID_ARG;
  if (meets_store(span(*K, p.kv_heads, n), *store) || meets_store(span(*V, p.kv_heads, n), *store) ||
      meets_store(span(rows, 4 * n), *store))
    return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_paged_append(p, *K, *V, rows, n, d, static_cast<cudaStream_t>(stream)));
}

h3kv_status h3kv_paged_read(const h3kv_paged_store *store, const int32_t *rows, int64_t n, const h3kv_rows *K,
                            const h3kv_rows *V, void *stream) {
  h3kv::PagedArgs p;
  h3kv_status st = paged_args(store, &p);
  if (st != H3KV_OK) return st;
  if (n < 0 || n > kMaxRows) return H3KV_ERR_INVALID_ARG;
  if (n == 0 || p.kv_heads == 0) return H3KV_OK;
  if (!out_rows_ok(K, p.kv_heads, n) || !out_rows_ok(V, p.kv_heads, n) || !rows || !aligned(rows, 4))
    return H3KV_ERR_INVALID_ARG;
  const Span k = span(*K, p.kv_heads, n), v = span(*V, p.kv_heads, n), r = span(rows, 4 * n);
  if (rows_meet(*K, *V, p.kv_heads, n) || meet(k, r) || meet(v, r) || meets_store(k, *store) || meets_store(v, *store))
    return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_paged_read(p, rows, n, *K, *V, d, static_cast<cudaStream_t>(stream)));
}

h3kv_status h3kv_paged_copy(const h3kv_paged_store *store, const int32_t *src, const int32_t *dst, int64_t n,
                            void *stream) {
  h3kv::PagedArgs p;
  h3kv_status st = paged_args(store, &p);
  if (st != H3KV_OK) return st;
  if (n < 0 || n > kMaxRows / 16) return H3KV_ERR_INVALID_ARG;
  if (n == 0 || p.kv_heads == 0) return H3KV_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return H3KV_ERR_INVALID_ARG;
  if (meets_store(span(src, 4 * n), *store) || meets_store(span(dst, 4 * n), *store)) return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_paged_copy(p, src, dst, n, static_cast<cudaStream_t>(stream)));
}

h3kv_status h3kv_paged_keep(const h3kv_paged_store *store, const int32_t *page_table, int64_t max_pages,
                            const int32_t *lengths, const int32_t *cu_nodes, int32_t seqs, const uint8_t *keep,
                            int64_t nodes, int32_t *new_lengths, void *stream) {
  h3kv::PagedArgs p;
  h3kv_status st = paged_args(store, &p);
  if (st != H3KV_OK) return st;
  if (seqs < 0 || seqs > kMaxSeqs || nodes < 0 || nodes > kMaxRows) return H3KV_ERR_INVALID_ARG;
  if (!table_ok(page_table, max_pages)) return H3KV_ERR_INVALID_ARG;
  if (seqs == 0) return H3KV_OK;
  if (!lengths || !cu_nodes || !new_lengths || (!keep && nodes > 0)) return H3KV_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(cu_nodes, 4) || !aligned(new_lengths, 4)) return H3KV_ERR_INVALID_ARG;
  // the others are read by every head's CTA while new_lengths is written
  const Span in[] = {span(lengths, 4ll * seqs), span(cu_nodes, 4ll * (seqs + 1)),
                     span(page_table, 4 * seqs * max_pages), span(keep, nodes)};
  if (meets_any(span(new_lengths, 4ll * seqs), in) || meets_store(span(new_lengths, 4ll * seqs), *store))
    return H3KV_ERR_INVALID_ARG;
  for (const Span &x : in)
    if (meets_store(x, *store)) return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_paged_keep(p, page_table, max_pages, lengths, cu_nodes, seqs, keep, nodes,
                                           new_lengths, static_cast<cudaStream_t>(stream)));
}

size_t h3kv_attend_tree_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t nodes, int32_t seqs) {
  if (q_heads < 0 || kv_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kMaxGroup || nodes < 0 ||
      nodes > kMaxRows || seqs < 0 || seqs > kMaxSeqs)
    return 0;
  return h3kv::tree_workspace_bytes(q_heads, kv_heads, nodes, seqs);
}

h3kv_status h3kv_attend_tree(const h3kv_rows *Q, int32_t q_heads, int64_t nodes, const h3kv_paged_store *store,
                             const int32_t *page_table, int64_t max_pages, const int32_t *lengths,
                             const int32_t *cu_nodes, int32_t seqs, const int32_t *parents, float softmax_scale,
                             const h3kv_rows *O, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  h3kv::TreeArgs a{};
  h3kv_status st = paged_args(store, &a.p);
  if (st != H3KV_OK) return st;
  if (q_heads < 0 || q_heads > kMaxHeads || nodes < 0 || seqs < 0 || seqs > kMaxSeqs) return H3KV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(q_heads) * nodes > kMaxRows) return H3KV_ERR_INVALID_ARG;
  if (!table_ok(page_table, max_pages)) return H3KV_ERR_INVALID_ARG;
  if (a.p.kv_heads < 1 || q_heads % a.p.kv_heads != 0 || q_heads / a.p.kv_heads > kMaxGroup)
    return H3KV_ERR_INVALID_ARG;
  if (q_heads == 0 || nodes == 0 || seqs == 0) return H3KV_OK;
  if (a.p.pages == 0 || max_pages == 0) return H3KV_ERR_INVALID_ARG;  // queries over an empty cache
  if (!rows_ok(Q, q_heads, nodes) || !out_rows_ok(O, q_heads, nodes)) return H3KV_ERR_INVALID_ARG;
  if (!lengths || !cu_nodes || !aligned(lengths, 4) || !aligned(cu_nodes, 4) || !aligned(parents, 4) ||
      !aligned(lse, 4))
    return H3KV_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 32) ||
      workspace_bytes < h3kv::tree_workspace_bytes(q_heads, a.p.kv_heads, nodes, seqs))
    return H3KV_ERR_INVALID_ARG;
  // what is written lies apart from the rest (O over Q is the caller's: a row of
  // Q has been read before that of O is written)
  const Span o = span(*O, q_heads, nodes), z = span(lse, 4 * q_heads * nodes),
             ws = span(workspace, static_cast<int64_t>(h3kv::tree_workspace_bytes(q_heads, a.p.kv_heads, nodes, seqs)));
  const Span in[] = {span(page_table, 4 * seqs * max_pages), span(lengths, 4ll * seqs), span(cu_nodes, 4ll * (seqs + 1)),
                     span(parents, 4 * nodes)};
  if (meet(o, z) || meet(o, ws) || meet(z, ws) || meet(z, span(*Q, q_heads, nodes)) ||
      meet(ws, span(*Q, q_heads, nodes)))
    return H3KV_ERR_INVALID_ARG;
  for (const Span &x : {o, z, ws})
    if (meets_any(x, in) || meets_store(x, *store)) return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  a.p.err = d.err;
  a.q = *Q;
  a.o = *O;
  a.lse = lse;
  a.page_table = page_table;
  a.lengths = lengths;
  a.cu_nodes = cu_nodes;
  a.parents = parents;
  a.max_pages = max_pages;
  a.nodes = nodes;
  a.q_heads = q_heads;
  a.group = q_heads / a.p.kv_heads;
  a.seqs = seqs;
  a.scale_log2 = scale_log2_of(softmax_scale);
  a.workspace = static_cast<float *>(workspace);
  a.ctas = d.num_sms;
  a.timeout_ns = d.timeout_ns;
  a.segment_timeout_ns = segment_timeout(d.timeout_ns, max_pages * a.p.page_size);
  a.withhold_p_tile1 = d.withhold_p_tile1;
  return status_of(h3kv::launch_attend_tree(a, static_cast<cudaStream_t>(stream)));
}

h3kv_status h3kv_attend_prompt(const h3kv_rows *Q, int32_t q_heads, int64_t q_rows, const h3kv_rows *K,
                               const h3kv_rows *V, int32_t kv_heads, int64_t k_rows, const int32_t *cu_q,
                               const int32_t *cu_k, int32_t seqs, int32_t causal, float softmax_scale,
                               const h3kv_rows *O, float *lse, void *stream) {
  if (q_heads < 0 || q_heads > kMaxHeads || kv_heads < 1 || q_heads % kv_heads != 0) return H3KV_ERR_INVALID_ARG;
  if (q_rows < 0 || k_rows < 0 || seqs < 0 || seqs > kMaxSeqs) return H3KV_ERR_INVALID_ARG;
  if (q_rows > kMaxRows / (q_heads > 0 ? q_heads : 1) || k_rows > kMaxRows / kv_heads) return H3KV_ERR_INVALID_ARG;
  if (q_heads == 0 || q_rows == 0 || seqs == 0) return H3KV_OK;
  if (!rows_ok(Q, q_heads, q_rows) || !out_rows_ok(O, q_heads, q_rows)) return H3KV_ERR_INVALID_ARG;
  if (k_rows > 0 && (!rows_ok(K, kv_heads, k_rows) || !rows_ok(V, kv_heads, k_rows))) return H3KV_ERR_INVALID_ARG;
  if (!cu_q || !cu_k || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return H3KV_ERR_INVALID_ARG;
  // what is written lies apart from the rest (O over Q, and O beside Q, K and V
  // in one buffer, is the caller's)
  const Span o = span(*O, q_heads, q_rows), z = span(lse, 4 * q_heads * q_rows);
  const Span cu[] = {span(cu_q, 4ll * (seqs + 1)), span(cu_k, 4ll * (seqs + 1))};
  if (meet(o, z) || meets_any(o, cu) || meets_any(z, cu) || meet(z, span(*Q, q_heads, q_rows)) ||
      (k_rows > 0 && (meet(z, span(*K, kv_heads, k_rows)) || meet(z, span(*V, kv_heads, k_rows)))))
    return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  const h3kv_status st = h3kv::serve_device(&d);
  if (st != H3KV_OK) return st;
  h3kv::PromptArgs a{};
  a.q = *Q;
  a.o = *O;
  if (k_rows > 0) {
    a.k = *K;
    a.v = *V;
  }
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.q_rows = q_rows;
  a.k_rows = k_rows;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.group = q_heads / kv_heads;
  a.seqs = seqs;
  a.causal = causal ? 1 : 0;
  a.scale_log2 = scale_log2_of(softmax_scale);
  a.err = d.err;
  a.timeout_ns = d.timeout_ns;
  a.segment_timeout_ns = segment_timeout(d.timeout_ns, k_rows);
  a.withhold_p_tile1 = d.withhold_p_tile1;
  a.num_sms = d.num_sms;
  return status_of(h3kv::launch_attend_prompt(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
