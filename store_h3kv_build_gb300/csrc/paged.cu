// paged.cu -- the paged kvi8r cache: rows written (rotated and quantised),
// read back, pages copied, drafted rows kept or dropped.
//
// All four are bound by HBM at size and by latency for a decoding step's few
// rows; none has arithmetic worth a tensor core.
#include "ptx.cuh"
#include "attend.cuh"
#include "serve_rows.cuh"
#include "store_fwht.cuh"

namespace h3kv {
namespace {

constexpr int kThreads = 256;

// Pool row `r` -> its row in [pages, kv_heads, page_size].
__device__ __forceinline__ int64_t pool_row(const PagedArgs &p, int32_t r, int32_t head) {
  return ((static_cast<int64_t>(r >> p.page_shift) * p.kv_heads + head) << p.page_shift) + (r & (p.page_size - 1));
}
// Pool row of token `t`, -1 if it is left out (or out of range, which is
// reported).
__device__ __forceinline__ int32_t row_of_token(const PagedArgs &p, const int32_t *__restrict__ rows, int64_t t,
                                                int64_t n) {
  const int32_t r = t < n ? __ldg(rows + t) : -1;
  if (r < p.pages * p.page_size) return r;
  atomicOr(p.err, kErrIndex);
  return -1;
}

// The tiles that a CTA walks: token tile x of y = 2 head + (V ? 1 : 0), from
// tile blockIdx.x in steps of gridDim.x.  (A 64-bit division for each tile was
// a third of the read kernel's instructions.)
constexpr int kTokens = 128;
struct TileWalk {
  int32_t x, y, tiles_x, tiles_y, dx, dy;
  __device__ __forceinline__ TileWalk(int64_t n, int32_t kv_heads, uint32_t first, uint32_t step) {
    tiles_x = static_cast<int32_t>((n + kTokens - 1) / kTokens);
    tiles_y = 2 * kv_heads;
    dx = static_cast<int32_t>(step % tiles_x);
    dy = static_cast<int32_t>(step / tiles_x);
    x = static_cast<int32_t>(first % tiles_x);
    y = static_cast<int32_t>(first / tiles_x);
  }
  __device__ __forceinline__ bool in() const { return y < tiles_y; }
  __device__ __forceinline__ int32_t token() const { return x * kTokens; }
  __device__ __forceinline__ int32_t head() const { return y >> 1; }
  __device__ __forceinline__ bool v() const { return y & 1; }
  __device__ __forceinline__ void next() {
    x += dx;
    y += dy;
    if (x >= tiles_x) {
      x -= tiles_x;
      ++y;
    }
  }
};

// ----------------------------------------------------------------- append --
// A persistent CTA walks 128-token tiles of one head of K or of V; a producer
// warp streams them into a ring with TMA (whatever the strides), and two
// threads share a row.  H128 = [[H64, H64], [H64, -H64]]: thread hf forms the
// sum (hf 0) or difference (hf 1) of the row's halves and transforms 64 values
// in registers, so a row costs no shuffle but the one for its absmax.  (With a
// row over 8 lanes, 48 shuffles for 4 rows, it ran at 3.5 TB/s.)  65536 rows of
// 8 heads: 71.5 us, 5.66 TB/s; 217088: 225 us, 5.96 TB/s; bound by HBM.
constexpr int kComputeWarps = 2 * kTokens / 32;
constexpr int kAppendThreads = 2 * kTokens + 32;
constexpr int kAppendStages = 3;
constexpr int kTokenTileBytes = kTokens * 256;

struct AppendSmem {
  uint8_t in[kAppendStages][kTokenTileBytes];
  uint64_t full[kAppendStages], empty[kAppendStages];
  int abort;
};
constexpr int kAppendSmemBytes = sizeof(AppendSmem) + 1024;

// Four codes rne(x m), clamped to [-127, 127], packed (the conversion packs
// and saturates from above; -128 is kept out before).
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float m) {
  const int ia = __float2int_rn(fmaxf(a * m, -127.f)), ib = __float2int_rn(fmaxf(b * m, -127.f));
  const int ic = __float2int_rn(fmaxf(c * m, -127.f)), id = __float2int_rn(fmaxf(d * m, -127.f));
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\t"
      "cvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\t"
      "cvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}"
      : "=r"(r)
      : "r"(ia), "r"(ib), "r"(ic), "r"(id));
  return r;
}

template <bool kWide>
__global__ void __launch_bounds__(kAppendThreads, 2)
    append_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const PagedArgs p, const int32_t *__restrict__ rows, const int64_t n, const uint64_t timeout_ns) {
  extern __shared__ uint8_t smem_raw[];
  AppendSmem &sm = *reinterpret_cast<AppendSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  TileWalk t(n, p.kv_heads, blockIdx.x, gridDim.x);
  if (tid == 0) {
    for (int s = 0; s < kAppendStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), kComputeWarps);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtx w{p.err, &sm.abort, timeout_ns};
  int slot = 0;
  uint32_t phase = 0;
  if (warp == kComputeWarps) {
    const uint32_t go = elect_one();
    int issued[kAppendStages] = {};
    for (; t.in(); t.next()) {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.empty[slot]), phase ^ 1u, w))) break;
      if (go) {
        const CUtensorMap *map = t.v() ? &tm_v : &tm_k;
        const uint32_t bar = smem_u32(&sm.full[slot]), dst = smem_u32(sm.in[slot]);
        mbar_arrive_expect_tx(bar, kTokenTileBytes);
        tma_load_3d(dst, map, 0, t.token(), t.head(), bar);
        tma_load_3d(dst + kTokenTileBytes / 2, map, 64, t.token(), t.head(), bar);
      }
      ++issued[slot];
      if (++slot == kAppendStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    // every copy that was issued must land before the CTA exits, also where a
    // row warp gives up behind the last of them
    for (int s = 0; s < kAppendStages; ++s)
      if (issued[s]) mbar_wait_drain(smem_u32(&sm.full[s]), (issued[s] - 1) & 1, kDrainNs);
    return;
  }
  const int i = tid >> 1, hf = tid & 1;  // row in the tile, half of the result
  const float2 sign = hf ? make_float2(-1.f, -1.f) : make_float2(1.f, 1.f);
  for (; t.in(); t.next()) {
    const int32_t r = row_of_token(p, rows, static_cast<int64_t>(t.token()) + i, n);
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.full[slot]), phase, w))) return;
    // 2^-7 first (exact), so that a sum of 128 of the largest bf16 values stays
    // finite; the values that it makes subnormal lie far below the least scale
    float x[64];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const uint32_t off = sw128_off(i, g);
      float lo[8], hi[8];
      unpack_bf16x8(*reinterpret_cast<const uint4 *>(sm.in[slot] + off), lo);
      unpack_bf16x8(*reinterpret_cast<const uint4 *>(sm.in[slot] + kTokenTileBytes / 2 + off), hi);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 k = make_float2(0.0078125f, 0.0078125f);
        const float2 a = __fmul2_rn(make_float2(lo[e], lo[e + 1]), k);
        const float2 b = __fmul2_rn(make_float2(hi[e], hi[e + 1]), k);
        const float2 s = __ffma2_rn(b, sign, a);
        x[8 * g + e] = s.x;
        x[8 * g + e + 1] = s.y;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
    if (++slot == kAppendStages) {
      slot = 0;
      phase ^= 1u;
    }
    fwht64_packed(x);
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < 64; ++e) a = fmaxf(a, fabsf(x[e]));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    // s = fp16(absmax(x H) / 127), saturated; codes rne(x H / s) with the stored
    // s.  absmax * sqrt(128) / 127 in two fp32 parts p + e: where p alone lies
    // on the tie between two fp16 values, e says which side the product is on.
    // On a tie the bits that fp16 drops (13, and one more for each power of two
    // below its least normal value 2^-14) are a one and zeros.
    constexpr float kHi = 0.08908431977033615f, kLo = -8.806923523785315e-10f;  // sqrt(128) / 127
    float scale = a * kHi;
    const float e = fmaf(a, kLo, fmaf(a, kHi, -scale));
    const uint32_t bits = __float_as_uint(scale);
    const int kept = min(19, static_cast<int>(bits >> 23) - 94);
    if (kept >= 8 && ((bits & 0x7FFFFFu) | 0x800000u) << kept == 0x80000000u)
      scale = __uint_as_float(bits + (e > 0.f ? 1 : e < 0.f ? -1 : 0));
    __half s = __float2half_rn(scale);
    if (__hisinf(s)) s = __ushort_as_half(0x7BFFu);
    // the maximum drops NaN: a row that holds one (every transformed value is
    // NaN then) says so by its scale
    if (x[0] != x[0]) s = __ushort_as_half(0x7FFFu);
    const float sf = __half2float(s);
    const float m = sf > 0.f ? kInvSqrt128 * 128.0f / sf : 0.f;
    if (r >= 0) {
      const int64_t at = pool_row(p, r, t.head());
      uint8_t *dst = reinterpret_cast<uint8_t *>(t.v() ? p.v_codes : p.k_codes) + at * 128 + hf * 64;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at4 = 32 * g + 4 * k;
          c[k] = code4(x[at4], x[at4 + 1], x[at4 + 2], x[at4 + 3], m);
        }
        if constexpr (kWide) {
          st_global_v8(dst + 32 * g, c);
        } else {
          reinterpret_cast<uint4 *>(dst)[2 * g] = make_uint4(c[0], c[1], c[2], c[3]);
          reinterpret_cast<uint4 *>(dst)[2 * g + 1] = make_uint4(c[4], c[5], c[6], c[7]);
        }
      }
      if (hf == 0) (t.v() ? p.v_scales : p.k_scales)[at] = __half_as_ushort(s);
    }
  }
}

// ------------------------------------------------------------------- read --
// Two threads share a row here too: each dequantises its 64 codes as the
// attention does (fp16(code * scale)) and transforms them, then the pair
// exchanges sums and differences (H128 = H2 x H64).  The next tile's codes, and
// the row numbers of the one after it, are loaded before the present one is
// worked on.
// A warp's 16 rows leave by TMA from a buffer of its own, two of them in turn:
// whole lines (written in 32-byte pieces from registers, 4.46 TB/s became 4.93).
// 65536 rows of 8 heads: 75.6 us, 5.35 TB/s; 217088: 237 us, 5.65 TB/s.  Codes
// brought to shared memory by asynchronous copies, three tiles ahead, were 3 %
// slower: more instructions for a tile, with 16 warps an SM that issue in
// 57 % of the cycles already.
constexpr int kReadRows = 16;                       // rows of a warp in a tile
constexpr int kReadHalfBytes = kReadRows * 128;     // 64 channels of them
constexpr int kReadSmemBytes = kThreads / 32 * 2 * 2 * kReadHalfBytes + 1024;

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 2)
    read_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const PagedArgs p, const int32_t *__restrict__ rows, const int64_t n) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *out = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) +
                 (threadIdx.x >> 5) * (4 * kReadHalfBytes);
  const int i = threadIdx.x >> 1, hf = threadIdx.x & 1, lane = threadIdx.x & 31;
  int buf = 0;
  struct Row {
    uint4 c[4];
    uint16_t s;
  };
  auto index = [&](const TileWalk &t) {
    return t.in() ? row_of_token(p, rows, static_cast<int64_t>(t.token()) + i, n) : -1;
  };
  auto load = [&](const TileWalk &t, int32_t r) {
    Row x;
    x.s = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) x.c[g] = make_uint4(0, 0, 0, 0);
    if (r >= 0) {
      const int64_t at = pool_row(p, r, t.head());
      const uint4 *src = reinterpret_cast<const uint4 *>((t.v() ? p.v_codes : p.k_codes) + at * 128) + hf * 4;
      if constexpr (kWide) {
        ld_global_v8(src, x.c[0], x.c[1]);
        ld_global_v8(src + 2, x.c[2], x.c[3]);
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) x.c[g] = src[g];
      }
      x.s = (t.v() ? p.v_scales : p.k_scales)[at];
    }
    return x;
  };
  TileWalk t(n, p.kv_heads, blockIdx.x, gridDim.x), ahead = t;
  Row next = load(t, index(t));
  ahead.next();
  int32_t r = index(ahead);
  for (; t.in(); t.next()) {
    const Row row = next;
    next = load(ahead, r);
    ahead.next();
    r = index(ahead);
    float x[64];
    const __half s = __ushort_as_half(row.s);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t h[8];
      attn::dequant16(row.c[g], __halves2half2(s, s), h);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
        x[16 * g + 2 * k] = f.x;
        x[16 * g + 2 * k + 1] = f.y;
      }
    }
    fwht64_packed(x);
    const float2 norm = make_float2(kInvSqrt128, kInvSqrt128);
    const float2 sign = hf ? make_float2(-1.f, -1.f) : make_float2(1.f, 1.f);
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
      const float2 v = __fmul2_rn(make_float2(x[e], x[e + 1]), norm);
      const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v.x, 1), __shfl_xor_sync(0xffffffffu, v.y, 1));
      const float2 z = __ffma2_rn(v, sign, o);  // lo + hi, or lo - hi in the second half
      x[e] = z.x;
      x[e + 1] = z.y;
    }
    // the buffer's store before last has read it
    if (lane == 0) bulk_wait_read<1>();
    __syncwarp();
    uint8_t *half = out + buf * (2 * kReadHalfBytes) + hf * kReadHalfBytes;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = pack_bf16x2(x[8 * g + 2 * k], x[8 * g + 2 * k + 1]);
      *reinterpret_cast<uint4 *>(half + sw128_off(lane >> 1, g)) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    const int32_t token = t.token() + (i & ~(kReadRows - 1));
    if (lane == 0) {
      if (token < n) {  // (rows from n on are not written: they lie outside the map)
        const CUtensorMap *map = t.v() ? &tm_v : &tm_k;
        const uint32_t src = smem_u32(out) + buf * (2 * kReadHalfBytes);
        tma_store_3d(map, src, 0, token, t.head());
        tma_store_3d(map, src + kReadHalfBytes, 64, token, t.head());
      }
      bulk_commit();
    }
    buf ^= 1;
  }
  if (lane == 0) bulk_wait_done();
}

// A page's codes (and scales) of all heads are contiguous: four block copies
// per page, cut into chunks of 16 KB, one CTA each.  Bound by HBM: 1500 pages of
// 64 rows and 8 heads 63.5 us, 6.29 TB/s; 24 pages 5.8 us, a call's latency.
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
// thread.  Bound by latency: four dependent loads and a store.
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
                                int64_t n, const ServeDevice &d, cudaStream_t stream) {
  CUtensorMap tk, tv;
  if (!encode_rows_bf16(&tk, K, p.kv_heads, n, kTokens) || !encode_rows_bf16(&tv, V, p.kv_heads, n, kTokens))
    return cudaErrorInvalidValue;
  // whole 32-byte sectors per store where the codes' alignment allows
  const bool wide = ((reinterpret_cast<uintptr_t>(p.k_codes) | reinterpret_cast<uintptr_t>(p.v_codes)) & 31) == 0;
  auto kernel = wide ? append_kernel<true> : append_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  const cudaError_t e = allow_smem(kernel, kAppendSmemBytes, allowed[wide]);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (n + kTokens - 1) / kTokens * p.kv_heads * 2;
  const unsigned grid = static_cast<unsigned>(tiles < 2 * d.num_sms ? tiles : 2 * d.num_sms);
  kernel<<<grid, kAppendThreads, kAppendSmemBytes, stream>>>(tk, tv, p, rows, n, d.timeout_ns);
  return cudaGetLastError();
}

cudaError_t launch_paged_read(const PagedArgs &p, const int32_t *rows, int64_t n, const h3kv_rows &K,
                              const h3kv_rows &V, const ServeDevice &d, cudaStream_t stream) {
  CUtensorMap tk, tv;
  if (!encode_rows_bf16(&tk, K, p.kv_heads, n, kReadRows) || !encode_rows_bf16(&tv, V, p.kv_heads, n, kReadRows))
    return cudaErrorInvalidValue;
  // whole 32-byte sectors per load where the codes' alignment allows
  const bool wide = ((reinterpret_cast<uintptr_t>(p.k_codes) | reinterpret_cast<uintptr_t>(p.v_codes)) & 31) == 0;
  auto kernel = wide ? read_kernel<true> : read_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  const cudaError_t e = allow_smem(kernel, kReadSmemBytes, allowed[wide]);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (n + kTokens - 1) / kTokens * p.kv_heads * 2;
  const unsigned grid = static_cast<unsigned>(tiles < 2 * d.num_sms ? tiles : 2 * d.num_sms);
  kernel<<<grid, kThreads, kReadSmemBytes, stream>>>(tk, tv, p, rows, n);
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
