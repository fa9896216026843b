// Host check of csrc/spans.h: rows_meet() of small strided tensors against a
// mark for every element, and spans at the ends of the address space.
#include <stdio.h>

#include <set>

#include "../store_h3kv_build_gb300/csrc/spans.h"

using namespace h3kv;

int main() {
  static uint16_t base[1];
  long cases = 0, wrong = 0, met = 0, apart_within = 0;
  const int64_t strides[] = {128, 136, 256, 264, 384, 512, 640, 768, 1024, 1280};
  for (int heads = 1; heads <= 4; ++heads)
    for (int rows = 1; rows <= 5; ++rows)
      for (int64_t hs : strides)
        for (int64_t rs : strides) {
          const h3kv_rows a{base, hs, rs};
          std::set<int64_t> mark;  // first elements of a's rows
          for (int h = 0; h < heads; ++h)
            for (int r = 0; r < rows; ++r) mark.insert(h * hs + r * rs);
          for (int64_t d = -5000; d <= 5000; d += 8) {
            const h3kv_rows b{reinterpret_cast<uint16_t *>(reinterpret_cast<uintptr_t>(base) + 2 * d), hs, rs};
            bool want = false;
            for (int h = 0; h < heads && !want; ++h)
              for (int r = 0; r < rows && !want; ++r) {
                const auto at = mark.upper_bound(d + h * hs + r * rs - 128);
                want = at != mark.end() && *at < d + h * hs + r * rs + 128;
              }
            const bool got = rows_meet(a, b, heads, rows);
            ++cases;
            met += want;
            wrong += got != want;
            apart_within += !want && meet(span(a, heads, rows), span(b, heads, rows));
          }
        }
  // strides of the largest accepted size do not wrap
  const h3kv_rows far{base, (1ll << 38) - 8, (1ll << 38) - 8};
  if (span(far, 65535, (1ll << 31) - 256).end != UINTPTR_MAX) ++wrong;
  if (span(far, 2, 1).end != reinterpret_cast<uintptr_t>(base) + 2 * ((1ull << 38) - 8 + 128)) ++wrong;
  if (meet(span(nullptr, 64), span(nullptr, 64))) ++wrong;  // an absent tensor
  if (meet(span(base + 8, 0), span(base, 64)) || meet(span(base, 64), span(base + 8, 0))) ++wrong;  // an empty one
  printf("cases %ld, meeting %ld, apart within each other's extent %ld, wrong %ld\n", cases, met, apart_within, wrong);
  return wrong != 0;
}
