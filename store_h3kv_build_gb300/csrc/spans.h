// spans.h -- which of a call's tensors lie over one another: host-side checks
// of the serving operators' outputs against what else the call reads or writes.
// Only host code.
#pragma once

#include <stdint.h>

#include "../../include/h3kv_serve.h"

namespace h3kv {

// Bytes of memory, saturated at the end of the address space.
struct Span {
  uintptr_t begin, end;
};
inline Span span(const void *p, __int128 bytes) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const __int128 last = static_cast<__int128>(at) + (p ? bytes : 0);
  return {at, last > static_cast<__int128>(UINTPTR_MAX) ? UINTPTR_MAX : static_cast<uintptr_t>(last)};
}
// Elements from the first to the last of [heads, rows, 128], gaps included.
inline __int128 extent(const h3kv_rows &r, int64_t heads, int64_t rows) {
  return (heads > 1 ? static_cast<__int128>(heads - 1) * r.head_stride : 0) +
         (rows > 1 ? static_cast<__int128>(rows - 1) * r.row_stride : 0) + H3KV_HEAD_DIM;
}
inline Span span(const h3kv_rows &r, int64_t heads, int64_t rows) { return span(r.data, 2 * extent(r, heads, rows)); }
inline bool meet(const Span &a, const Span &b) {
  return a.begin < b.end && b.begin < a.end && a.begin < a.end && b.begin < b.end;
}
template <int kN>
inline bool meets_any(const Span &a, const Span (&others)[kN]) {
  for (const Span &o : others)
    if (meet(a, o)) return true;
  return false;
}
// Whether a span lies over one of a store's four buffers.
inline bool meets_store(const Span &a, const h3kv_paged_store &st) {
  const int64_t rows = static_cast<int64_t>(st.pages) * st.kv_heads * st.page_size;
  const Span of[] = {span(st.k_codes, rows * H3KV_HEAD_DIM), span(st.v_codes, rows * H3KV_HEAD_DIM),
                     span(st.k_scales, rows * 2), span(st.v_scales, rows * 2)};
  return meets_any(a, of);
}

// Whether two tensors [heads, rows, 128] share an element.  Exact where their
// strides are equal, as those of two that take turns in one buffer are; else
// by their extents.
inline bool rows_meet(const h3kv_rows &a, const h3kv_rows &b, int64_t heads, int64_t rows) {
  if (!meet(span(a, heads, rows), span(b, heads, rows))) return false;
  if ((heads > 1 && a.head_stride != b.head_stride) || (rows > 1 && a.row_stride != b.row_stride)) return true;
  const __int128 d = (static_cast<__int128>(reinterpret_cast<uintptr_t>(b.data)) - reinterpret_cast<uintptr_t>(a.data)) / 2;
  // an element of each meet where |d + x head_stride + y row_stride| < 128 for
  // some |x| < heads, |y| < rows: all steps of the shorter axis, and of the
  // other those next to the sum's zero
  const bool by_head = heads <= rows;
  const int64_t n = by_head ? heads : rows, m = by_head ? rows : heads;
  const int64_t sn = n > 1 ? (by_head ? a.head_stride : a.row_stride) : 0;
  const int64_t sm = m > 1 ? (by_head ? a.row_stride : a.head_stride) : 0;
  for (int64_t x = 1 - n; x < n; ++x) {
    const __int128 at = d + static_cast<__int128>(x) * sn, zero = sm > 0 ? -at / sm : 0;
    for (__int128 y = zero - 1; y <= zero + 1; ++y) {
      const __int128 off = at + y * sm;
      if (y > -m && y < m && off > -H3KV_HEAD_DIM && off < H3KV_HEAD_DIM) return true;
    }
  }
  return false;
}

}  // namespace h3kv
