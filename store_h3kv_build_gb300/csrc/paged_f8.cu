// paged_f8.cu -- the paged e4m3 cache: rows rotated and written, read back, pages
// copied.  Bound by HBM at size and by latency for a decoding step's few rows.
#include "block_scan.cuh"
#include "paged_f8.cuh"

namespace h3kv {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;


// The sequence of token t: the last with cu[i] <= t; -1 if t belongs to none.
__device__ __forceinline__ int seq_of(const BatchArgs &b, int64_t t) {
  int lo = 0, hi = b.seqs;  // cu[lo] <= t < cu[hi], if the counts rise
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(b.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return __ldg(b.cu + lo) <= t && t < __ldg(b.cu + lo + 1) ? lo : -1;
}

// A warp takes 4 rows of Q, 8 lanes each.
template <int kMode>
__device__ __forceinline__ void rotate_q(const PagedF8Args &p, const RotateArgs &r, const BatchArgs &b, int64_t unit) {
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int64_t x = unit * 4 + (lane >> 3), total = r.n * r.q_heads;
  const int64_t t = x < total ? x / r.q_heads : 0;
  const int h = x < total ? static_cast<int>(x - t * r.q_heads) : 0;
  const int i = x < total ? seq_of(b, t) : -1;
  bool on = i >= 0;
  int64_t pos = 0;
  if (on) {
    const BatchCounts c = batch_counts(b, p.page_shift, r.n, i);
    on = !c.bad;
    pos = on ? angle_row(r, r.positions ? __ldg(r.positions + t) : c.len - c.m + (t - c.c0), p.err) : 0;
  }
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  Angles<kMode> a;
  a.load(r, pos, l);
  if (on) {
    const uint4 *src = row_at(r.q, h, t, l);
    lo = src[0];
    hi = src[8];
  }
  float y[16];
  rotate_lane<kMode, false>(lo, hi, a, r.dim, y);
  if (on) {
    uint4 *dst = row_out(r.q_out, h, t, l);
    dst[0] = pack_bf16x8(y);
    dst[8] = pack_bf16x8(y + 8);
  }
}

// New rows of a sequence and of a head of K (pair 2 h) or of V (2 h + 1), from token `lo`
// on: of that token's page, or all where they are no more than a page's.
struct NewRows {
  int32_t seq, lo;  // seq -1: none
  int32_t c0, m, len;
  uint32_t pair;
};

// One warp writes them, page by page: once over the page's rows for the largest value, once
// for the codes.  (16 rows at once, loads and angles of all of them under way, took
// registers for 170 a thread: 28 us.)
template <int kMode, bool kKeys>
__device__ __forceinline__ void append_pages(const PagedF8Args &p, const RotateArgs &r, const BatchArgs &b,
                                             const NewRows &c) {
  const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3, h = c.pair >> 1;
  const int32_t p0 = c.len - c.m, end = c.m <= p.page_size ? c.len : min(c.len, (c.lo & ~(p.page_size - 1)) + p.page_size);
  uint8_t *codes = kKeys ? p.k_codes : p.v_codes;
  float *scales = kKeys ? p.k_scales : p.v_scales;
  const h3kv_rows &in = kKeys ? r.k : r.v;
  for (int32_t lo = c.lo, hi; lo < end; lo = hi) {
    const int32_t begin = lo & ~(p.page_size - 1);
    hi = min(begin + p.page_size, end);
    const int32_t page = batch_page(b, p, c.seq, lo);
    const int64_t at = static_cast<int64_t>(page) * p.kv_heads + h;
    uint8_t *base = codes + (at << p.page_shift) * 128;
    float y[16];
    auto get = [&](int32_t j) {
      const int32_t pos = min(j, hi - 1);
      const int64_t t = static_cast<int64_t>(c.c0) + (pos - p0);
      const uint4 *src = row_at(in, h, t, l);
      const uint4 a = src[0], z = src[8];
      if constexpr (kKeys && kMode != kRotNone) {
        Angles<kMode> ang;
        ang.load(r, angle_row(r, r.positions ? __ldg(r.positions + t) : pos, p.err), l);
        rotate_lane<kMode, true>(a, z, ang, r.dim, y);
      } else {
        unpack_bf16x8(a, y);
        unpack_bf16x8(z, y + 8);
      }
    };
    float top = 0.f;
#pragma unroll 1
    for (int32_t j = lo; j < hi; j += 4) {
      get(j + sub);
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(y[e]));
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    int e = f8_exponent(top);
    if (page >= 0 && lo > begin) {
      const float old = scales[at];
      e = max(e, f8_scale_exponent(old));
      const float m = old * exp2i(-e);
      if (m != 1.f) {
        for (int k = lane; k < (lo - begin) * 8; k += 32) {
          uint4 w = reinterpret_cast<uint4 *>(base)[k];
          w = make_uint4(f8_recode4(w.x, m), f8_recode4(w.y, m), f8_recode4(w.z, m), f8_recode4(w.w, m));
          reinterpret_cast<uint4 *>(base)[k] = w;
        }
      }
    }
    const float m = exp2i(-e);
#pragma unroll 1
    for (int32_t j = lo; j < hi; j += 4) {
      if (hi - lo > 4) get(j + sub);  // (up to 4 rows are still there)
      __syncwarp();  // (K_out may be K: every lane's part of the row has been read)
      if (j + sub < hi) {
        if (page >= 0) {
          uint2 *dst = reinterpret_cast<uint2 *>(base + (j + sub - begin) * 128) + l;
          dst[0] = f8_codes8(y, m);
          dst[8] = f8_codes8(y + 8, m);
        }
        if (kKeys && r.k_out.data) {
          uint4 *dst = row_out(r.k_out, h, static_cast<int64_t>(c.c0) + (j + sub - p0), l);
          dst[0] = pack_bf16x8(y);
          dst[8] = pack_bf16x8(y + 8);
        }
      }
    }
    __syncwarp();
    if (page >= 0 && lane == 0) scales[at] = exp2i(e);
  }
}

// What the blocks of append_few_kernel do: `first` of them begin the new rows of each
// sequence, a warp for each head of K or of V; `later` take the pages behind a sequence's
// first where it has more new tokens than a page; the rest rotate Q.  A page depends
// on nothing in the pages before it, so that a chunk beside single tokens is not one
// warp's work: 63 tokens and a chunk of 2048, 32 and 8 heads, 41 us (875 so), 127 and one
// of 8192 71 us (3878), 31 and one of 512 39 us (224).
//
// Places of later pages: from 2 cu[i] >> shift on for sequence i.  One of m tokens, more
// than a page's, has at most (m - 2 >> shift) + 1 such pages, which is no more than the
// 2 m >> shift places that it has at least.  A lane each of a block's first warp looks for
// the page at one of `span` places, by bisection; the warps share those that there are.
// (Counts that fall, which is reported, may hide pages of other sequences.)
struct FewBlocks {
  uint32_t first, later;
  int32_t span;
};

// The page at a place.
__device__ __forceinline__ NewRows later_page(const PagedF8Args &p, const BatchArgs &b, int64_t n, int64_t place) {
  auto begin = [&](int i) { return 2 * static_cast<int64_t>(__ldg(b.cu + i)) >> p.page_shift; };
  int lo = 0, hi = b.seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (begin(mid) <= place) lo = mid;
    else hi = mid;
  }
  const int64_t k = place - begin(lo);
  const BatchCounts c = batch_counts(b, p.page_shift, n, lo);
  const int64_t at = (((c.len - c.m) >> p.page_shift) + 1 + k) << p.page_shift;
  const bool on = k >= 0 && c.m > p.page_size && at < c.len;
  return {on ? lo : -1, static_cast<int32_t>(at), static_cast<int32_t>(c.c0), c.m, c.len, 0};
}

// A block's share of the later pages.  A function of its own: inlined, it took the
// registers of the kernel from 64 to 84, and 4096 single tokens 72 us for 66.
template <int kMode>
__device__ __noinline__ void append_later(const PagedF8Args &p, const RotateArgs &r, const BatchArgs &b, uint32_t x,
                                          int32_t span) {
  __shared__ NewRows pages[32];
  __shared__ int found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    const uint32_t pairs = 2 * p.kv_heads, group = x / pairs;
    NewRows page = {-1};
    if (lane < span) page = later_page(p, b, r.n, static_cast<int64_t>(group) * span + lane);
    page.pair = x - group * pairs;
    const uint32_t on = __ballot_sync(0xffffffffu, page.seq >= 0);
    if (page.seq >= 0) pages[__popc(on & ((1u << lane) - 1))] = page;
    if (lane == 0) found = __popc(on);
  }
  __syncthreads();
#pragma unroll 1
  for (int k = warp; k < found; k += kWarps) {
    if (pages[k].pair & 1) append_pages<kMode, false>(p, r, b, pages[k]);
    else append_pages<kMode, true>(p, r, b, pages[k]);
  }
}

// Bound by latency: one token each of 1 to 64 sequences, 32 and 8 heads, 3.4 - 4 us, of 256
// 6.8.  Blocks an SM, by the registers of a rotation's angles and partners.
template <int kMode>
__global__ void __launch_bounds__(kThreads, kMode == kRotNone || kMode == kRotHalves128 ? 4 : 2)
    append_few_kernel(const __grid_constant__ PagedF8Args p, const __grid_constant__ RotateArgs r,
                      const __grid_constant__ BatchArgs b, const FewBlocks blocks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= blocks.first + blocks.later) {
    const int64_t unit = static_cast<int64_t>(blockIdx.x - blocks.first - blocks.later) * kWarps + warp;
    if constexpr (kMode != kRotNone) {
      if (unit * 4 < r.n * r.q_heads) rotate_q<kMode>(p, r, b, unit);
    }
    return;
  }
  if (blockIdx.x >= blocks.first) {
    append_later<kMode>(p, r, b, blockIdx.x - blocks.first, blocks.span);
    return;
  }
  const uint32_t pairs = 2 * p.kv_heads;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp, i = w / pairs;
  if (i >= b.seqs) return;
  const BatchCounts c = batch_counts(b, p.page_shift, r.n, static_cast<int>(i));
  const NewRows page = {static_cast<int32_t>(i), c.len - c.m, static_cast<int32_t>(c.c0), c.m, c.len,
                        static_cast<uint32_t>(w - i * pairs)};
  if (c.bad && page.pair == 0 && lane == 0) atomicOr(p.err, kErrIndex);
  if (page.pair & 1) append_pages<kMode, false>(p, r, b, page);
  else append_pages<kMode, true>(p, r, b, page);
}

// Many new tokens: a block takes windows of kTokens positions of a sequence, whole
// pages of it, a warp 4 tokens, 8 lanes each.  The lanes keep their tokens' angles
// while the block goes through the steps of the window: the heads of K, of V and
// of Q.  Bound by HBM; a step's rows are loaded under the step before (three steps
// before, through shared memory, was slower: 336 us against 319 with the read).  A
// page's largest value comes from its warps through shared memory, one barrier a
// step.  The steps of all windows are split evenly over the blocks.  65536 tokens of
// 32 and 8 heads: 247 us, 5.97 TB/s; 13 chunks of up to 3000, 16 and 4 heads: 34 us, of
// which 4 are the counts and the first rows.
template <int kMode, int kTokens>
__global__ void __launch_bounds__(kTokens * 8, kTokens == 64 && kMode != kRotHalves ? 2 : 1)
    append_many_kernel(const PagedF8Args p, const RotateArgs r, const BatchArgs b) {
  constexpr int kBlock = kTokens * 8, kBlockWarps = kBlock / 32;
  __shared__ int64_t scratch[kBlockWarps];
  __shared__ float tops[2][kBlockWarps];
  __shared__ struct {
    int64_t before;  // units before it
    BatchCounts c;
    int seq;
  } start;  // the block's first sequence
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane & 7;
  const int steps = 2 * p.kv_heads + r.q_heads;
  auto units_of = [&](const BatchCounts &c) -> int64_t {
    return c.m > 0 ? static_cast<int64_t>((c.len - 1) / kTokens - (c.len - c.m) / kTokens + 1) * steps : 0;
  };
  BatchCounts c = {};
  int64_t total = 0, at = 0, units = 0;  // at: units before this thread's sequence
  auto count = [&](int base, int64_t before) {
    c = {};
    if (base + tid < b.seqs) c = batch_counts(b, p.page_shift, r.n, base + tid);
    units = units_of(c);
    int64_t all;
    at = before + block_prefix<kBlock>(scratch, units, &all);
    return all;
  };
  for (int base = 0; base < b.seqs; base += kBlock) {
    total += count(base, total);
    if (c.bad && blockIdx.x == 0) atomicOr(p.err, kErrIndex);
  }
  int64_t u = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  if (u >= end) return;
  // the sequence that holds unit u: known already where one round covered them all
  int64_t before = 0;
  for (int base = 0; base < b.seqs; base += kBlock) {
    if (b.seqs > kBlock) before += count(base, before);
    if (u >= at && u < at + units) {
      start.before = at;
      start.seq = base + tid;
      start.c = c;
    }
    if (b.seqs > kBlock && u < before) break;
  }
  __syncthreads();
  before = start.before;
  int seq = start.seq, buf = 0;
  c = start.c;
  while (u < end) {
    units = units_of(c);
    if (u >= before + units) {
      before += units;
      c = batch_counts(b, p.page_shift, r.n, ++seq);
      continue;
    }
    const int32_t p0 = c.len - c.m, w = static_cast<int32_t>((u - before) / steps);
    const int first = static_cast<int>((u - before) - static_cast<int64_t>(w) * steps);
    const int last = static_cast<int>(end - u < steps - first ? first + (end - u) : steps);
    u += last - first;
    const int32_t at0 = (p0 / kTokens + w) * kTokens, pos = at0 + warp * 4 + (lane >> 3);
    const bool live = pos >= p0 && pos < c.len;
    const int64_t t = live ? c.c0 + (pos - p0) : 0;
    const int32_t begin = pos & ~(p.page_size - 1);  // the page's first token
    // any new token in the page, and tokens that it holds already
    const bool in = begin + p.page_size > p0 && begin < c.len, old_page = in && begin < p0;
    const int32_t page = in ? batch_page(b, p, seq, pos < c.len ? pos : c.len - 1) : -1;
    Angles<kMode> ang;
    ang.load(r, kMode != kRotNone && live ? angle_row(r, r.positions ? __ldg(r.positions + t) : pos, p.err) : 0, l);
    auto source = [&](int step) {
      return step < p.kv_heads       ? row_at(r.k, step, t, l)
             : step < 2 * p.kv_heads ? row_at(r.v, step - p.kv_heads, t, l)
                                     : row_at(r.q, step - 2 * p.kv_heads, t, l);
    };
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (live) {
      const uint4 *src = source(first);
      lo = src[0];
      hi = src[8];
    }
    for (int step = first; step < last; ++step) {
      uint4 next_lo = make_uint4(0, 0, 0, 0), next_hi = next_lo;
      if (live && step + 1 < last) {
        const uint4 *src = source(step + 1);
        next_lo = src[0];
        next_hi = src[8];
      }
      float y[16];
      if (step >= 2 * p.kv_heads) {
        if constexpr (kMode != kRotNone) {
          rotate_lane<kMode, false>(lo, hi, ang, r.dim, y);
          if (live) {
            uint4 *dst = row_out(r.q_out, step - 2 * p.kv_heads, t, l);
            dst[0] = pack_bf16x8(y);
            dst[8] = pack_bf16x8(y + 8);
          }
        }
      } else {
        const bool keys = step < p.kv_heads;
        const int h = keys ? step : step - p.kv_heads;
        if (keys) {
          rotate_lane<kMode, true>(lo, hi, ang, r.dim, y);
          if (live && r.k_out.data) {
            uint4 *dst = row_out(r.k_out, h, t, l);
            dst[0] = pack_bf16x8(y);
            dst[8] = pack_bf16x8(y + 8);
          }
        } else {
          unpack_bf16x8(lo, y);
          unpack_bf16x8(hi, y + 8);
        }
        float top = 0.f;  // (rows that are not live hold zeros)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(y[e]));
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        if (lane == 0) tops[buf][warp] = top;
        uint8_t *codes = keys ? p.k_codes : p.v_codes;
        float *scales = keys ? p.k_scales : p.v_scales;
        const int64_t at = static_cast<int64_t>(page) * p.kv_heads + h;
        // (read by every warp of the page before one of them writes the new one)
        const float old = old_page && page >= 0 ? scales[at] : 0.f;
        __syncthreads();
        const int of_page = p.page_size >> 2, w0 = warp & ~(of_page - 1);
        top = tops[buf][w0 + (lane & (of_page - 1))];
        buf ^= 1;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        int e = f8_exponent(top);
        if (page >= 0) {
          uint2 *dst = reinterpret_cast<uint2 *>(codes + ((at << p.page_shift) + (pos - begin)) * 128) + l;
          if (old_page) {
            e = max(e, f8_scale_exponent(old));
            const float m = old * exp2i(-e);
            if (m != 1.f && pos < p0) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint2 x = dst[8 * k];
                dst[8 * k] = make_uint2(f8_recode4(x.x, m), f8_recode4(x.y, m));
              }
            }
          }
          const float m = exp2i(-e);
          if (live) {
            dst[0] = f8_codes8(y, m);
            dst[8] = f8_codes8(y + 8, m);
          }
          if (warp == w0 && lane == 0) scales[at] = exp2i(e);
        }
      }
      lo = next_lo;
      hi = next_hi;
    }
  }
}

// Eight lanes take a row of K or of V, 16 codes each.  Bound by HBM: 65536 rows of 8
// heads 71 us, 5.7 TB/s; 217088: 227 us, 5.9 TB/s.
__global__ void __launch_bounds__(kThreads)
    read_kernel(const PagedF8Args p, const int32_t *__restrict__ rows, const int64_t n, const h3kv_rows K,
                const h3kv_rows V) {
  const int l = threadIdx.x & 7;
  const int64_t total = n * p.kv_heads * 2;
  for (int64_t x = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 3; x < total;
       x += static_cast<int64_t>(gridDim.x) * (kThreads / 8)) {
    const int64_t hv = x / n, t = x - hv * n;
    const int h = static_cast<int>(hv >> 1), v = static_cast<int>(hv & 1);
    const int32_t row = __ldg(rows + t);
    const bool bad = row >= p.pages * p.page_size;
    if (bad && l == 0) atomicOr(p.err, kErrIndex);
    uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row >= 0 && !bad) {
      const int64_t at = static_cast<int64_t>(row >> p.page_shift) * p.kv_heads + h;
      const uint4 w = reinterpret_cast<const uint4 *>((v ? p.v_codes : p.k_codes) +
                                                      ((at << p.page_shift) + (row & (p.page_size - 1))) * 128)[l];
      const __half2 s = __float2half2_rn((v ? p.v_scales : p.k_scales)[at]);
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t f = e4m3x2_to_f16x2(k & 1 ? in[k >> 1] >> 16 : in[k >> 1] & 0xFFFFu);
        const float2 g = __half22float2(__hmul2(*reinterpret_cast<const __half2 *>(&f), s));
        o[k] = pack_bf16x2(g.x, g.y);
      }
    }
    uint4 *dst = reinterpret_cast<uint4 *>((v ? V : K).data + h * (v ? V : K).head_stride + t * (v ? V : K).row_stride) + 2 * l;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// A page's codes of all heads are contiguous, and so are its scales: chunks of
// 16 KB, one CTA each; the first of K and of V takes the scales along.  1500 pages of
// 64 rows and 8 heads 61 us, 6.5 TB/s.
__global__ void __launch_bounds__(kThreads)
    copy_kernel(const PagedF8Args p, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                const uint32_t chunks) {
  const uint32_t i = blockIdx.x / (2 * chunks), c = blockIdx.x - i * 2 * chunks;
  const int32_t from = __ldg(src + i), to = __ldg(dst + i);
  if (from < 0 || to < 0) return;
  if (from >= p.pages || to >= p.pages) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
    return;
  }
  const int64_t bytes = (static_cast<int64_t>(p.kv_heads) << p.page_shift) * 128;
  uint8_t *codes = c & 1 ? p.v_codes : p.k_codes;
  const int64_t at = static_cast<int64_t>(c >> 1) * kCopyChunk;
  const uint8_t *s = codes + from * bytes + at;
  uint8_t *d = codes + to * bytes + at;
  const int len = static_cast<int>(bytes - at < kCopyChunk ? bytes - at : kCopyChunk);  // a multiple of 16
  uint4 w[kCopyChunk / 16 / kThreads];
#pragma unroll
  for (int k = 0; k < kCopyChunk / 16 / kThreads; ++k) {
    const int o = (k * kThreads + threadIdx.x) * 16;
    if (o < len) w[k] = __ldcs(reinterpret_cast<const uint4 *>(s + o));
  }
#pragma unroll
  for (int k = 0; k < kCopyChunk / 16 / kThreads; ++k) {
    const int o = (k * kThreads + threadIdx.x) * 16;
    if (o < len) *reinterpret_cast<uint4 *>(d + o) = w[k];
  }
  if (c < 2) {
    float *scales = c & 1 ? p.v_scales : p.k_scales;
    for (int h = threadIdx.x; h < p.kv_heads; h += kThreads)
      scales[static_cast<int64_t>(to) * p.kv_heads + h] = scales[static_cast<int64_t>(from) * p.kv_heads + h];
  }
}

}  // namespace

namespace {

// The blocks of append_few_kernel.  A block's warps have a place each while that takes no
// more than four blocks an SM.
FewBlocks few_blocks(const PagedF8Args &p, const BatchArgs &b, int64_t n, int32_t num_sms) {
  const int64_t pairs = 2 * static_cast<int64_t>(p.kv_heads), places = (2 * n >> p.page_shift) + 1;
  FewBlocks f = {};
  f.first = static_cast<uint32_t>((b.seqs * pairs + kWarps - 1) / kWarps);
  for (f.span = kWarps; f.span < 32 && (places + f.span - 1) / f.span * pairs > 4 * num_sms;) f.span *= 2;
  if (n > p.page_size) f.later = static_cast<uint32_t>((places + f.span - 1) / f.span * pairs);
  return f;
}

// Which of the two kernels is sooner done, by what they take (32 and 8 heads, pages
// of 64): a warp of the one for few goes through a page's tokens, or a short sequence's, in
// 0.42 us each behind a start of 3.5, and through as many pages as its group of places
// has for each warp; all warps through 6600 rows of K, V and Q a microsecond; a block
// of the other takes 1.5 us a step where windows are full, 2.5 where they are not, behind
// 6 us.  Measured, tokens of each sequence, few and many: 1 x 4 3.6 and 5.6, 1 x 12 7.9 and
// 6.0, 1 x 64 30 and 7.5; 16 x 12 7.7 and 13, 16 x 64 31 and 19 (pages of 16: 14.5 and
// 18); 64 x 16 10 and 38, 64 x 64 36 and 41; 256 x 1 6 and 44, 256 x 64 115 and 108.
// The host knows no more than the mean: where single tokens hide a chunk, its pages take the
// one for few up to a whole page's time (39 us for 31 tokens and a chunk of 512).
bool many_tokens(int64_t n, int64_t seqs, int64_t steps, int64_t page, int64_t window, int64_t blocks) {
  const double mean = static_cast<double>(n) / seqs, rows = static_cast<double>(n) * steps;
  const double alone = 3.5 + 0.42 * (mean < page ? mean : page), all = 2.5 + rows / 6600, few = alone > all ? alone : all;
  const double per_block = (static_cast<double>(n) / window + seqs) * steps / blocks;
  return few > 6.0 + (mean >= window ? 1.5 : 2.5) * per_block;
}

template <int kMode>
cudaError_t launch_append(const PagedF8Args &p, const RotateArgs &r, const BatchArgs &b, const ServeDevice &d,
                          cudaStream_t stream) {
  const int window = p.page_size <= 64 ? 64 : 128, blocks = d.num_sms * (window == 64 && kMode != kRotHalves ? 2 : 1);
  const FewBlocks f = few_blocks(p, b, r.n, d.num_sms);
  if (many_tokens(r.n, b.seqs, 2 * p.kv_heads + r.q_heads, p.page_size * f.span / kWarps, window, blocks)) {
    if (window == 64) append_many_kernel<kMode, 64><<<blocks, 512, 0, stream>>>(p, r, b);
    else append_many_kernel<kMode, 128><<<blocks, 1024, 0, stream>>>(p, r, b);
    return cudaGetLastError();
  }
  const int64_t q_units = kMode != kRotNone ? (r.n * r.q_heads + 3) / 4 : 0;
  const int64_t grid = f.first + static_cast<int64_t>(f.later) + (q_units + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  append_few_kernel<kMode><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(p, r, b, f);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_append_f8(const PagedF8Args &p, const RotateArgs &r, const BatchArgs &b, const ServeDevice &d,
                             cudaStream_t stream) {
  switch (r.mode) {
    case kRotNone: return launch_append<kRotNone>(p, r, b, d, stream);
    case kRotHalves128: return launch_append<kRotHalves128>(p, r, b, d, stream);
    case kRotHalves: return launch_append<kRotHalves>(p, r, b, d, stream);
    default: return launch_append<kRotPairs>(p, r, b, d, stream);
  }
}

cudaError_t launch_read_f8(const PagedF8Args &p, const int32_t *rows, int64_t n, const h3kv_rows &K,
                           const h3kv_rows &V, const ServeDevice &d, cudaStream_t stream) {
  const int64_t blocks = (n * p.kv_heads * 2 + kThreads / 8 - 1) / (kThreads / 8);
  const unsigned grid = static_cast<unsigned>(blocks < 8 * d.num_sms ? blocks : 8 * d.num_sms);
  read_kernel<<<grid, kThreads, 0, stream>>>(p, rows, n, K, V);
  return cudaGetLastError();
}

cudaError_t launch_copy_f8(const PagedF8Args &p, const int32_t *src, const int32_t *dst, int64_t n,
                           cudaStream_t stream) {
  const int64_t blocks = copy_f8_blocks(p);
  copy_kernel<<<static_cast<unsigned>(n * blocks), kThreads, 0, stream>>>(p, src, dst,
                                                                        static_cast<uint32_t>(blocks / 2));
  return cudaGetLastError();
}

}  // namespace h3kv
