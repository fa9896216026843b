// paged.cu -- the paged kvi8r cache: rows written (rotated and quantised),
// read back, pages copied, drafted rows kept or dropped.
//
// All four are bound by HBM at size and by latency for a decoding step's few
// rows; none has arithmetic worth a tensor core.
#include "ptx.cuh"
#include "serve_rows.cuh"

namespace h3kv {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = kThreads / 8;

// Pool row `r` -> its row in [pages, kv_heads, page_size].
__device__ __forceinline__ int64_t pool_row(const PagedArgs &p, int32_t r, int32_t head) {
  return ((static_cast<int64_t>(r >> p.page_shift) * p.kv_heads + head) << p.page_shift) + (r & (p.page_size - 1));
}

// What a CTA works on: 32 tokens of one head of K or of V.
struct Piece {
  int64_t token;
  int32_t head;
  bool v;
};
__device__ __forceinline__ Piece piece_of(int64_t n, int32_t kv_heads) {
  const uint32_t groups = static_cast<uint32_t>((n + kRowsPerCta - 1) / kRowsPerCta);
  const uint32_t b = blockIdx.x, y = b / groups;
  return {static_cast<int64_t>(b - y * groups) * kRowsPerCta + (threadIdx.x >> 3), static_cast<int32_t>(y >> 1),
          (y & 1) != 0};
}

__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float m) {
  auto q = [m](float x) {
    const int v = __float2int_rn(x * m);
    return static_cast<uint32_t>(v > 127 ? 127 : v < -127 ? -127 : v) & 0xFFu;
  };
  return q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
}

// A warp takes 4 rows, 8 lanes each: 32 bytes of a row per thread, one
// 16-bit scale per row, 16 code bytes per thread.
__global__ void __launch_bounds__(kThreads)
    append_kernel(const PagedArgs p, const h3kv_rows K, const h3kv_rows V, const int32_t *__restrict__ rows,
                  const int64_t n) {
  const Piece w = piece_of(n, p.kv_heads);
  const int l = threadIdx.x & 7;
  int32_t r = -1;
  if (w.token < n) r = __ldg(rows + w.token);
  if (r >= p.pages * p.page_size) {
    if (l == 0) atomicOr(p.err, kErrIndex);
    r = -1;
  }
  const h3kv_rows &in = w.v ? V : K;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (r >= 0) {
    const uint4 *src =
        reinterpret_cast<const uint4 *>(in.data + w.head * in.head_stride + w.token * in.row_stride) + l;
    lo = __ldcs(src);
    hi = __ldcs(src + 8);
  }
  float x[16];
  unpack_bf16x8(lo, x);
  unpack_bf16x8(hi, x + 8);
  // 2^-7 first (exact), so that a sum of 128 of the largest bf16 values stays
  // finite; the values that it makes subnormal lie far below the least scale
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] *= 0.0078125f;
  fwht128_oct(x, l);
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  // s = fp16(absmax(x H) / 127), saturated; codes rne(x H / s) with the stored s.
  // absmax * sqrt(128) / 127 in two fp32 parts p + e: where p alone lies on
  // the tie between two fp16 values, e says which side the product is on.
  constexpr float kHi = 0.08908431977033615f, kLo = -8.806923523785315e-10f;  // sqrt(128) / 127
  float scale = a * kHi;
  const float e = fmaf(a, kLo, fmaf(a, kHi, -scale));
  uint32_t bits = __float_as_uint(scale);
  if ((bits & 0x1FFFu) == 0x1000u) scale = __uint_as_float(bits + (e > 0.f ? 1 : e < 0.f ? -1 : 0));
  __half s = __float2half_rn(scale);
  if (__hisinf(s)) s = __ushort_as_half(0x7BFFu);
  const float sf = __half2float(s);
  const float m = sf > 0.f ? kInvSqrt128 * 128.0f / sf : 0.f;
  if (r >= 0) {
    const int64_t at = pool_row(p, r, w.head);
    uint2 *dst = reinterpret_cast<uint2 *>((w.v ? p.v_codes : p.k_codes) + at * 128) + l;
    dst[0] = make_uint2(code4(x[0], x[1], x[2], x[3], m), code4(x[4], x[5], x[6], x[7], m));
    dst[8] = make_uint2(code4(x[8], x[9], x[10], x[11], m), code4(x[12], x[13], x[14], x[15], m));
    if (l == 0) (w.v ? p.v_scales : p.k_scales)[at] = __half_as_ushort(s);
  }
}

// The inverse: 16 code bytes per thread, dequantised as the attention does
// (fp16(code * scale)), un-rotated in fp32 and rounded to bf16 once.
__global__ void __launch_bounds__(kThreads)
    read_kernel(const PagedArgs p, const int32_t *__restrict__ rows, const int64_t n, const h3kv_rows K,
                const h3kv_rows V) {
  const Piece w = piece_of(n, p.kv_heads);
  const int l = threadIdx.x & 7;
  int32_t r = -1;
  if (w.token < n) r = __ldg(rows + w.token);
  if (r >= p.pages * p.page_size) {
    if (l == 0) atomicOr(p.err, kErrIndex);
    r = -1;
  }
  uint2 c[2] = {make_uint2(0, 0), make_uint2(0, 0)};
  __half s = __ushort_as_half(0);
  if (r >= 0) {
    const int64_t at = pool_row(p, r, w.head);
    const uint2 *src = reinterpret_cast<const uint2 *>((w.v ? p.v_codes : p.k_codes) + at * 128) + l;
    c[0] = src[0];
    c[1] = src[8];
    s = __ushort_as_half((w.v ? p.v_scales : p.k_scales)[at]);
  }
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t word = (i & 4) ? c[i >> 3].y : c[i >> 3].x;
    const int code = static_cast<int8_t>(word >> ((i & 3) * 8));
    x[i] = __half2float(__hmul(__int2half_rn(code), s));
  }
  fwht128_oct(x, l);
  if (w.token < n) {
    const h3kv_rows &out = w.v ? V : K;
    uint4 *dst = reinterpret_cast<uint4 *>(out.data + w.head * out.head_stride + w.token * out.row_stride) + l;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= kInvSqrt128;
    dst[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                        pack_bf16x2(x[6], x[7]));
    dst[8] = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                        pack_bf16x2(x[14], x[15]));
  }
}

// A page's codes (and scales) of all heads are contiguous: four block copies
// per page, cut into chunks of 16 KB, one CTA each.
constexpr int kCopyChunk = 16384;

__global__ void __launch_bounds__(kThreads)
    copy_kernel(const PagedArgs p, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                const uint32_t code_chunks, const uint32_t scale_chunks) {
  const uint32_t per_page = 2 * (code_chunks + scale_chunks);
  const uint32_t i = blockIdx.x / per_page;
  uint32_t c = blockIdx.x - i * per_page;
  const int32_t from = __ldg(src + i), to = __ldg(dst + i);
  if (from < 0 || to < 0) return;
  if (from >= p.pages || to >= p.pages) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
    return;
  }
  const bool v = c & 1;
  c >>= 1;
  const bool scales = c >= code_chunks;
  const int64_t rows = static_cast<int64_t>(p.kv_heads) << p.page_shift;
  const int64_t bytes = scales ? rows * 2 : rows * 128;
  uint8_t *base = scales ? reinterpret_cast<uint8_t *>(v ? p.v_scales : p.k_scales)
                         : reinterpret_cast<uint8_t *>(v ? p.v_codes : p.k_codes);
  const int64_t at = static_cast<int64_t>(scales ? c - code_chunks : c) * kCopyChunk;
  const uint8_t *s = base + from * bytes + at;
  uint8_t *d = base + to * bytes + at;
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
}

// One CTA for a sequence and head.  A row may move onto one that is itself
// kept and moves on, so every kept row is read into registers before any is
// written: 64 rows x 2 tensors x 8 granules of 16 bytes = 1024, four per
// thread.
__global__ void __launch_bounds__(kThreads)
    keep_kernel(const PagedArgs p, const int32_t *__restrict__ table, const int64_t max_pages,
                const int32_t *__restrict__ lengths, const int32_t *__restrict__ cu, const uint8_t *__restrict__ keep,
                const int64_t nodes, int32_t *__restrict__ new_lengths) {
  constexpr int kMax = H3KV_TREE_MAX_NODES;
  __shared__ int64_t row_of[kMax];  // of node j: its row in [pages, kv_heads, page_size]
  __shared__ uint8_t kept[kMax];    // the kept nodes, in order
  __shared__ uint32_t half_count[2];
  const int heads = p.kv_heads > 0 ? p.kv_heads : 1;
  const int i = blockIdx.x / heads, head = blockIdx.x - i * heads;
  const int tid = threadIdx.x;
  const int32_t len = __ldg(lengths + i), c0 = __ldg(cu + i), c1 = __ldg(cu + i + 1);
  const int64_t m64 = static_cast<int64_t>(c1) - c0;
  const bool ok = c0 >= 0 && m64 >= 0 && m64 <= kMax && c1 <= nodes && len >= m64 &&
                  len <= (max_pages << p.page_shift);
  if (!ok) {
    if (tid == 0 && head == 0) {
      atomicOr(p.err, kErrIndex);
      new_lengths[i] = len;
    }
    return;
  }
  const int m = static_cast<int>(m64);
  if (tid < kMax) {
    bool bad = false;
    if (tid < m) {
      const int32_t pos = len - m + tid;
      const int32_t page = __ldg(table + i * max_pages + (pos >> p.page_shift));
      bad = page < 0 || page >= p.pages;
      row_of[tid] = bad ? -1
                        : ((static_cast<int64_t>(page) * p.kv_heads + head) << p.page_shift) +
                              (pos & (p.page_size - 1));
    }
    if (bad) atomicOr(p.err, kErrIndex);
    const bool k = tid < m && keep[c0 + tid] != 0;
    const uint32_t votes = __ballot_sync(0xffffffffu, k);
    if ((tid & 31) == 0) half_count[tid >> 5] = __popc(votes);
    named_bar_sync(1, kMax);
    if (k) kept[(tid >= 32 ? half_count[0] : 0) + __popc(votes & ((1u << (tid & 31)) - 1))] = tid;
  }
  __syncthreads();
  const int n = static_cast<int>(half_count[0] + half_count[1]);
  if (tid == 0 && head == 0) new_lengths[i] = len - m + n;
  if (p.kv_heads == 0) return;
  uint4 w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int u = k * kThreads + tid, rank = u >> 4;
    if (rank < n && kept[rank] != rank) {
      const int64_t from = row_of[kept[rank]];
      if (from >= 0)
        w[k] = reinterpret_cast<const uint4 *>(((u & 8) ? p.v_codes : p.k_codes) + from * 128)[u & 7];
    }
  }
  uint16_t sc = 0;
  const int srank = tid >> 1;
  uint16_t *scales = (tid & 1) ? p.v_scales : p.k_scales;
  const bool smove = srank < n && kept[srank < kMax ? srank : 0] != srank;
  if (smove && row_of[kept[srank]] >= 0) sc = scales[row_of[kept[srank]]];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int u = k * kThreads + tid, rank = u >> 4;
    if (rank < n && kept[rank] != rank && row_of[kept[rank]] >= 0 && row_of[rank] >= 0)
      reinterpret_cast<uint4 *>(((u & 8) ? p.v_codes : p.k_codes) + row_of[rank] * 128)[u & 7] = w[k];
  }
  if (smove && row_of[kept[srank]] >= 0 && row_of[srank] >= 0) scales[row_of[srank]] = sc;
}

bool grid_of(int64_t a, int64_t b, int64_t c, unsigned *out) {
  if (a > INT32_MAX || b > INT32_MAX / a || c > INT32_MAX / (a * b)) return false;
  *out = static_cast<unsigned>(a * b * c);
  return true;
}

}  // namespace

cudaError_t launch_paged_append(const PagedArgs &p, const h3kv_rows &K, const h3kv_rows &V, const int32_t *rows,
                                int64_t n, cudaStream_t stream) {
  unsigned grid;
  if (!grid_of((n + kRowsPerCta - 1) / kRowsPerCta, p.kv_heads, 2, &grid)) return cudaErrorInvalidValue;
  append_kernel<<<grid, kThreads, 0, stream>>>(p, K, V, rows, n);
  return cudaGetLastError();
}

cudaError_t launch_paged_read(const PagedArgs &p, const int32_t *rows, int64_t n, const h3kv_rows &K,
                              const h3kv_rows &V, cudaStream_t stream) {
  unsigned grid;
  if (!grid_of((n + kRowsPerCta - 1) / kRowsPerCta, p.kv_heads, 2, &grid)) return cudaErrorInvalidValue;
  read_kernel<<<grid, kThreads, 0, stream>>>(p, rows, n, K, V);
  return cudaGetLastError();
}

cudaError_t launch_paged_copy(const PagedArgs &p, const int32_t *src, const int32_t *dst, int64_t n,
                              cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.kv_heads) << p.page_shift;
  const int64_t codes = (rows * 128 + kCopyChunk - 1) / kCopyChunk, scales = (rows * 2 + kCopyChunk - 1) / kCopyChunk;
  unsigned grid;
  if (!grid_of(n, codes + scales, 2, &grid)) return cudaErrorInvalidValue;
  copy_kernel<<<grid, kThreads, 0, stream>>>(p, src, dst, static_cast<uint32_t>(codes),
                                             static_cast<uint32_t>(scales));
  return cudaGetLastError();
}

cudaError_t launch_paged_keep(const PagedArgs &p, const int32_t *page_table, int64_t max_pages,
                              const int32_t *lengths, const int32_t *cu_nodes, int32_t seqs, const uint8_t *keep,
                              int64_t nodes, int32_t *new_lengths, cudaStream_t stream) {
  unsigned grid;
  if (!grid_of(seqs, p.kv_heads > 0 ? p.kv_heads : 1, 1, &grid)) return cudaErrorInvalidValue;
  keep_kernel<<<grid, kThreads, 0, stream>>>(p, page_table, max_pages, lengths, cu_nodes, keep, nodes, new_lengths);
  return cudaGetLastError();
}

}  // namespace h3kv
