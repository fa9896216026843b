// serve_f8.h -- internal launchers behind h3kv_serve_f8.h (not part of the public
// header).  As in serve.h, arguments have been checked and index arrays are
// checked by the kernels.
#pragma once

#include "../../include/h3kv_serve_f8.h"
#include "serve.h"

namespace h3kv {

// How channels are paired: not at all, c with c + 64, c with c + dim / 2 in
// general, neighbours.
enum RotationMode : int32_t { kRotNone, kRotHalves128, kRotHalves, kRotPairs };

// Rows that are rotated, and where to.
struct RotateArgs {
  h3kv_rows q, q_out, k, v, k_out;  // k_out.data NULL: not wanted
  const float *table;
  const int32_t *positions;
  int64_t table_rows, n;
  int32_t dim, mode, q_heads;
};

struct PagedF8Args {
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  int32_t pages, kv_heads, page_size, page_shift;
  uint32_t *err;
};

// A batch of sequences over a page table.
struct BatchArgs {
  const int32_t *page_table, *lengths, *cu;
  int64_t max_pages;
  int32_t seqs;
};

cudaError_t launch_append_rotated(const PagedArgs &p, const RotateArgs &r, const int32_t *rows, const ServeDevice &d,
                                  cudaStream_t stream);
cudaError_t launch_append_f8(const PagedF8Args &p, const RotateArgs &r, const BatchArgs &b, const ServeDevice &d,
                             cudaStream_t stream);
cudaError_t launch_read_f8(const PagedF8Args &p, const int32_t *rows, int64_t n, const h3kv_rows &K,
                           const h3kv_rows &V, const ServeDevice &d, cudaStream_t stream);
// Blocks that copy a page: chunks of 16 KB of its codes of K and of V.
constexpr int kCopyChunk = 16384;
inline int64_t copy_f8_blocks(const PagedF8Args &p) {
  const int64_t bytes = (static_cast<int64_t>(p.kv_heads) << p.page_shift) * 128;
  return 2 * ((bytes + kCopyChunk - 1) / kCopyChunk);
}
cudaError_t launch_copy_f8(const PagedF8Args &p, const int32_t *src, const int32_t *dst, int64_t n,
                           cudaStream_t stream);

struct AttendF8Args {
  PagedF8Args p;
  BatchArgs b;
  h3kv_rows q, o;
  float *lse;
  int64_t n;
  int32_t q_heads, group;
  float scale_log2;
  float *workspace;
  int32_t num_sms;
  uint64_t timeout_ns, segment_timeout_ns;
  int32_t withhold_p_tile1;
};
size_t attend_f8_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t n, int32_t seqs);
cudaError_t launch_attend_paged_f8(const AttendF8Args &a, cudaStream_t stream);

}  // namespace h3kv
