// serve_f8_abi.cu -- the C ABI of h3kv_serve_f8.h: host-side argument checks and
// the launches.
#include "serve_checks.h"
#include "serve_f8.h"

namespace {

using h3kv::BatchArgs;
using h3kv::meet;
using h3kv::meets_any;
using h3kv::PagedF8Args;
using h3kv::RotateArgs;
using h3kv::rows_meet;
using h3kv::same_rows;
using h3kv::Span;
using h3kv::span;
using namespace h3kv::checks;

// Sizes that a store may have: row numbers, and rows of all heads, in 31 bits.
bool store_sizes_ok(int32_t pages, int32_t kv_heads, int32_t page_size) {
  return pages >= 0 && kv_heads >= 0 && kv_heads <= kMaxHeads && page_shift_of(page_size) &&
         static_cast<int64_t>(pages) * page_size <= kMaxRows / (kv_heads > 0 ? kv_heads : 1);
}

h3kv_status paged_f8_args(const h3kv_paged_store_f8 *st, PagedF8Args *out) {
  if (!st || st->pages < 0 || st->kv_heads < 0 || st->kv_heads > kMaxHeads) return H3KV_ERR_INVALID_ARG;
  if (st->head_dim != H3KV_HEAD_DIM) return H3KV_ERR_UNSUPPORTED;
  const int32_t ps = st->page_size;
  if (!store_sizes_ok(st->pages, st->kv_heads, ps)) return H3KV_ERR_INVALID_ARG;
  if (st->pages > 0 && st->kv_heads > 0) {
    if (!st->k_codes || !st->v_codes || !st->k_scales || !st->v_scales) return H3KV_ERR_INVALID_ARG;
    if (!aligned(st->k_codes, 16) || !aligned(st->v_codes, 16) || !aligned(st->k_scales, 16) ||
        !aligned(st->v_scales, 16))
      return H3KV_ERR_INVALID_ARG;
  }
  *out = {st->k_codes, st->v_codes, st->k_scales, st->v_scales, st->pages, st->kv_heads, ps, page_shift_of(ps), nullptr};
  return H3KV_OK;
}

// The four buffers of a store of either kind.
struct StoreSpans {
  Span of[4];
  bool meets(const Span &a) const { return meets_any(a, of); }
};
StoreSpans store_spans(const PagedF8Args &p) {
  const __int128 heads = static_cast<__int128>(p.pages) * p.kv_heads, codes = heads * p.page_size * H3KV_HEAD_DIM;
  return {{span(p.k_codes, codes), span(p.v_codes, codes), span(p.k_scales, heads * 4), span(p.v_scales, heads * 4)}};
}
StoreSpans store_spans(const h3kv::PagedArgs &p) {
  const __int128 rows = static_cast<__int128>(p.pages) * p.kv_heads * p.page_size;
  return {{span(p.k_codes, rows * H3KV_HEAD_DIM), span(p.v_codes, rows * H3KV_HEAD_DIM), span(p.k_scales, rows * 2),
           span(p.v_scales, rows * 2)}};
}

// Q, K, V and their rotation: types, strides, and which of them lie over one
// another or over `others` (the call's index arrays) or the store.
h3kv_status rotate_args(const h3kv_rows *Q, int32_t q_heads, const h3kv_rows *Q_out, const h3kv_rows *K,
                        const h3kv_rows *V, const h3kv_rows *K_out, const h3kv_rotation *rot, const int32_t *positions,
                        int64_t n, int32_t kv_heads, const StoreSpans &store, const Span (&index)[4], RotateArgs *out) {
  if (!rows_ok(K, kv_heads, n) || !rows_ok(V, kv_heads, n)) return H3KV_ERR_INVALID_ARG;
  if (q_heads > 0 && (!rows_ok(Q, q_heads, n) || !out_rows_ok(Q_out, q_heads, n))) return H3KV_ERR_INVALID_ARG;
  if (K_out && !out_rows_ok(K_out, kv_heads, n)) return H3KV_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return H3KV_ERR_INVALID_ARG;
  *out = {};
  out->k = *K;
  out->v = *V;
  out->n = n;
  out->mode = h3kv::kRotNone;
  Span table = {};
  if (!rot) {
    if (q_heads > 0 || K_out || positions) return H3KV_ERR_INVALID_ARG;
  } else {
    if (rot->dim < 16 || rot->dim > H3KV_HEAD_DIM || rot->dim % 16 != 0 || rot->rows < 1 || rot->rows > kMaxRows ||
        !rot->table || !aligned(rot->table, 16))
      return H3KV_ERR_INVALID_ARG;
    table = span(rot->table, static_cast<__int128>(rot->rows) * rot->dim * 4);
    out->table = rot->table;
    out->table_rows = rot->rows;
    out->dim = rot->dim;
    out->positions = positions;
    out->mode = rot->interleaved            ? h3kv::kRotPairs
                : rot->dim == H3KV_HEAD_DIM ? h3kv::kRotHalves128
                                            : h3kv::kRotHalves;
  }
  const Span k = span(*K, kv_heads, n), v = span(*V, kv_heads, n);
  if (store.meets(k) || store.meets(v) || store.meets(table) || store.meets(span(positions, 4 * n)))
    return H3KV_ERR_INVALID_ARG;
  for (const Span &x : index)
    if (store.meets(x)) return H3KV_ERR_INVALID_ARG;
  auto out_ok = [&](const Span &o) {
    return !store.meets(o) && !meet(o, table) && !meet(o, span(positions, 4 * n)) && !meets_any(o, index);
  };
  if (q_heads > 0) {
    const Span q = span(*Q, q_heads, n), qo = span(*Q_out, q_heads, n);
    if (store.meets(q) || !out_ok(qo)) return H3KV_ERR_INVALID_ARG;
    if (!same_rows(*Q, *Q_out, q_heads, n) && rows_meet(*Q, q_heads, *Q_out, q_heads, n)) return H3KV_ERR_INVALID_ARG;
    if (rows_meet(*K, kv_heads, *Q_out, q_heads, n) || rows_meet(*V, kv_heads, *Q_out, q_heads, n))
      return H3KV_ERR_INVALID_ARG;
    out->q = *Q;
    out->q_out = *Q_out;
    out->q_heads = q_heads;
  }
  if (K_out) {
    if (!out_ok(span(*K_out, kv_heads, n))) return H3KV_ERR_INVALID_ARG;
    if (!same_rows(*K, *K_out, kv_heads, n) && rows_meet(*K, kv_heads, *K_out, kv_heads, n)) return H3KV_ERR_INVALID_ARG;
    if (rows_meet(*V, kv_heads, *K_out, kv_heads, n)) return H3KV_ERR_INVALID_ARG;
    if (q_heads > 0 && (rows_meet(*Q, q_heads, *K_out, kv_heads, n) || rows_meet(*Q_out, q_heads, *K_out, kv_heads, n)))
      return H3KV_ERR_INVALID_ARG;
    out->k_out = *K_out;
  }
  return H3KV_OK;
}

// Sequences over a page table.
h3kv_status batch_args(const int32_t *page_table, int64_t max_pages, const int32_t *lengths, const int32_t *cu,
                       int32_t seqs, BatchArgs *out) {
  if (seqs < 0 || seqs > kMaxSeqs || !table_ok(page_table, max_pages)) return H3KV_ERR_INVALID_ARG;
  if (seqs > 0 && (!lengths || !cu || !aligned(lengths, 4) || !aligned(cu, 4))) return H3KV_ERR_INVALID_ARG;
  *out = {page_table, lengths, cu, max_pages, seqs};
  return H3KV_OK;
}

}  // namespace

extern "C" {

h3kv_status h3kv_paged_append_rotated(const h3kv_rows *Q, int32_t q_heads, const h3kv_rows *Q_out,
                                      const h3kv_rows *K, const h3kv_rows *V, const h3kv_rows *K_out,
                                      const h3kv_rotation *rotation, const int32_t *positions, const int32_t *rows,
                                      int64_t n, const h3kv_paged_store *store, void *stream) {
  h3kv::PagedArgs p;
  h3kv_status st = paged_args(store, &p);
  if (st != H3KV_OK) return st;
  if (n < 0 || q_heads < 0 || q_heads > kMaxHeads || n > kMaxRows / (q_heads > 0 ? q_heads : 1) ||
      n > kMaxRows / (p.kv_heads > 0 ? p.kv_heads : 1))
    return H3KV_ERR_INVALID_ARG;
  if (n == 0 || (p.kv_heads == 0 && q_heads == 0)) return H3KV_OK;
  if (p.kv_heads == 0) return H3KV_ERR_INVALID_ARG;  // queries beside no cache
  if (!rotation || !positions || !rows || !aligned(rows, 4)) return H3KV_ERR_INVALID_ARG;
  RotateArgs r;
  const Span index[4] = {span(rows, 4 * n), {}, {}, {}};
  st = rotate_args(Q, q_heads, Q_out, K, V, K_out, rotation, positions, n, p.kv_heads, store_spans(p), index, &r);
  if (st != H3KV_OK) return st;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_append_rotated(p, r, rows, d, static_cast<cudaStream_t>(stream)));
}

size_t h3kv_paged_store_f8_bytes(int32_t pages, int32_t kv_heads, int32_t page_size, int32_t head_dim) {
  if (head_dim != H3KV_HEAD_DIM || !store_sizes_ok(pages, kv_heads, page_size)) return 0;
  return static_cast<size_t>(2) * static_cast<size_t>(pages) * static_cast<size_t>(kv_heads) *
         (static_cast<size_t>(page_size) * H3KV_HEAD_DIM + sizeof(float));
}

h3kv_status h3kv_paged_append_f8(const h3kv_rows *Q, int32_t q_heads, const h3kv_rows *Q_out, const h3kv_rows *K,
                                 const h3kv_rows *V, const h3kv_rows *K_out, const h3kv_rotation *rotation,
                                 const int32_t *positions, int64_t n, const h3kv_paged_store_f8 *store,
                                 const int32_t *page_table, int64_t max_pages, const int32_t *lengths,
                                 const int32_t *cu_new, int32_t seqs, void *stream) {
  PagedF8Args p;
  BatchArgs b;
  h3kv_status st = paged_f8_args(store, &p);
  if (st != H3KV_OK) return st;
  if ((st = batch_args(page_table, max_pages, lengths, cu_new, seqs, &b)) != H3KV_OK) return st;
  if (n < 0 || q_heads < 0 || q_heads > kMaxHeads || n > kMaxRows / (q_heads > 0 ? q_heads : 1) ||
      n > kMaxRows / (p.kv_heads > 0 ? p.kv_heads : 1))
    return H3KV_ERR_INVALID_ARG;
  if (n == 0 || seqs == 0 || (p.kv_heads == 0 && q_heads == 0)) return H3KV_OK;
  if (p.kv_heads == 0) return H3KV_ERR_INVALID_ARG;  // queries beside no cache
  RotateArgs r;
  const Span index[4] = {span(page_table, 4 * static_cast<__int128>(seqs) * max_pages), span(lengths, 4ll * seqs),
                         span(cu_new, 4ll * (seqs + 1)), {}};
  st = rotate_args(Q, q_heads, Q_out, K, V, K_out, rotation, positions, n, p.kv_heads, store_spans(p), index, &r);
  if (st != H3KV_OK) return st;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_append_f8(p, r, b, d, static_cast<cudaStream_t>(stream)));
}

h3kv_status h3kv_paged_read_f8(const h3kv_paged_store_f8 *store, const int32_t *rows, int64_t n, const h3kv_rows *K,
                               const h3kv_rows *V, void *stream) {
  PagedF8Args p;
  h3kv_status st = paged_f8_args(store, &p);
  if (st != H3KV_OK) return st;
  if (n < 0 || n > kMaxRows) return H3KV_ERR_INVALID_ARG;
  if (n == 0 || p.kv_heads == 0) return H3KV_OK;
  if (!out_rows_ok(K, p.kv_heads, n) || !out_rows_ok(V, p.kv_heads, n) || !rows || !aligned(rows, 4))
    return H3KV_ERR_INVALID_ARG;
  const Span k = span(*K, p.kv_heads, n), v = span(*V, p.kv_heads, n), r = span(rows, 4 * n);
  const StoreSpans of = store_spans(p);
  if (rows_meet(*K, *V, p.kv_heads, n) || meet(k, r) || meet(v, r) || of.meets(k) || of.meets(v))
    return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_read_f8(p, rows, n, *K, *V, d, static_cast<cudaStream_t>(stream)));
}

h3kv_status h3kv_paged_copy_f8(const h3kv_paged_store_f8 *store, const int32_t *src, const int32_t *dst, int64_t n,
                               void *stream) {
  PagedF8Args p;
  h3kv_status st = paged_f8_args(store, &p);
  if (st != H3KV_OK) return st;
  if (n < 0 || n > kMaxRows / 16) return H3KV_ERR_INVALID_ARG;
  if (n == 0 || p.kv_heads == 0) return H3KV_OK;
  if (n > INT32_MAX / h3kv::copy_f8_blocks(p)) return H3KV_ERR_INVALID_ARG;  // a launch's blocks
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return H3KV_ERR_INVALID_ARG;
  const StoreSpans of = store_spans(p);
  if (of.meets(span(src, 4 * n)) || of.meets(span(dst, 4 * n))) return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  p.err = d.err;
  return status_of(h3kv::launch_copy_f8(p, src, dst, n, static_cast<cudaStream_t>(stream)));
}

size_t h3kv_attend_paged_f8_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t n, int32_t seqs) {
  if (q_heads < 0 || kv_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kMaxGroup || n < 0 ||
      n > H3KV_PAGED_MAX_ROWS || seqs < 0 || seqs > kMaxSeqs)
    return 0;
  return h3kv::attend_f8_workspace_bytes(q_heads, kv_heads, n, seqs);
}

h3kv_status h3kv_attend_paged_f8(const h3kv_rows *Q, int32_t q_heads, int64_t n, const h3kv_paged_store_f8 *store,
                                 const int32_t *page_table, int64_t max_pages, const int32_t *lengths,
                                 const int32_t *cu_q, int32_t seqs, float softmax_scale, const h3kv_rows *O,
                                 float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  h3kv::AttendF8Args a{};
  h3kv_status st = paged_f8_args(store, &a.p);
  if (st != H3KV_OK) return st;
  if ((st = batch_args(page_table, max_pages, lengths, cu_q, seqs, &a.b)) != H3KV_OK) return st;
  if (q_heads < 0 || q_heads > kMaxHeads || n < 0 || n > H3KV_PAGED_MAX_ROWS) return H3KV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(q_heads) * n > kMaxRows) return H3KV_ERR_INVALID_ARG;
  if (a.p.kv_heads < 1 || q_heads % a.p.kv_heads != 0 || q_heads / a.p.kv_heads > kMaxGroup)
    return H3KV_ERR_INVALID_ARG;
  if (q_heads == 0 || n == 0 || seqs == 0) return H3KV_OK;
  if (a.p.pages == 0 || max_pages == 0) return H3KV_ERR_INVALID_ARG;  // queries over an empty cache
  if (!rows_ok(Q, q_heads, n) || !out_rows_ok(O, q_heads, n) || !aligned(lse, 4)) return H3KV_ERR_INVALID_ARG;
  const size_t need = h3kv::attend_f8_workspace_bytes(q_heads, a.p.kv_heads, n, seqs);
  if (!workspace || !aligned(workspace, 32) || workspace_bytes < need) return H3KV_ERR_INVALID_ARG;
  // what is written lies apart from the rest (O over Q is the caller's)
  const Span o = span(*O, q_heads, n), z = span(lse, 4 * q_heads * n), q = span(*Q, q_heads, n),
             ws = span(workspace, static_cast<__int128>(need));
  const Span in[] = {span(page_table, 4 * static_cast<__int128>(seqs) * max_pages), span(lengths, 4ll * seqs),
                     span(cu_q, 4ll * (seqs + 1))};
  const StoreSpans of = store_spans(a.p);
  if (meet(o, z) || meet(o, ws) || meet(z, ws) || meet(z, q) || meet(ws, q)) return H3KV_ERR_INVALID_ARG;
  for (const Span &x : {o, z, ws})
    if (meets_any(x, in) || of.meets(x)) return H3KV_ERR_INVALID_ARG;
  h3kv::ServeDevice d;
  if ((st = h3kv::serve_device(&d)) != H3KV_OK) return st;
  a.p.err = d.err;
  a.q = *Q;
  a.o = *O;
  a.lse = lse;
  a.n = n;
  a.q_heads = q_heads;
  a.group = q_heads / a.p.kv_heads;
  a.scale_log2 = scale_log2_of(softmax_scale);
  a.workspace = static_cast<float *>(workspace);
  a.num_sms = d.num_sms;
  a.timeout_ns = d.timeout_ns;
  a.segment_timeout_ns = segment_timeout(d.timeout_ns, max_pages * a.p.page_size);
  a.withhold_p_tile1 = d.withhold_p_tile1;
  return status_of(h3kv::launch_attend_paged_f8(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
