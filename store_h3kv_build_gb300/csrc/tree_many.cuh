// tree_many.cuh -- attention of drafted tokens over the paged kvi8r cache, and of
// new tokens over the paged e4m3 cache (kF8): the kernel for many rows of a
// sequence and kv head (the tcgen05 pipeline of serve_attend.cuh), the join, and
// the choice of kernel.
//
// Bound by shared memory, which feeds the products and carries the codes and
// their fp16 values, and by the issue slots that dequantisation and softmax
// share: 1.9 us for 256 rows over a 128-key tile, where the products alone take
// 1.3 (the tensor rate) and the bytes 0.75.  A segment costs some 12 us more
// before its first tile (counts, query rows, first page) and 4 behind its last.
// A thread spills 56 bytes (e4m3: 92).  Measured at 64 nodes, 32 query heads over 8: 2 x
// 131072 cached rows 228 us (1207 TFLOP/s), 32 x 8192 247 us, 128 x 2048 315 us,
// 512 x 512 453 us; 16 over 4 heads: 133, 138, 176 and 244 us.
//
// e4m3: K's codes go to the products as they are (kind::f8f6f4), with a row of Q as the
// sum of two e4m3 parts, which costs QK what fp16 does; V's are dequantised.  A tile
// takes 1.7 us for 256 rows, of which the products 1.65: 0.86 us for PV and QK of 128
// rows, where the best that cuBLAS reaches would be 0.69 (both operands of QK come from
// shared memory, 128 bytes a cycle, beside V's dequantisation).  V's products start at
// half of a tile's weights (460 -> 422 us for 16384 tokens).  16384 tokens, 8 heads over
// 2: 422 us (1300 TFLOP/s); 4 sequences of up to 16384 with up to 700 new tokens 158 us
// (1180); 32 heads over 8 and 32 x 8192 rows: 64 rows 140 us, 256 rows 213.  A segment
// costs 4 us beside its tiles: its last tile's mask, the output (2.1 us of the softmax
// warps), the next one's query rows.
// Weights by a polynomial in place of some of the ex2 were slower (434 us for an
// eighth of them); so was a join in this kernel (cooperative, by
// flags: 431 us, and 160 -> 168).
#pragma once

#include "store_fwht.cuh"
#include "tree.cuh"

namespace h3kv {
namespace serve {
namespace {

// e4m3: K's scales of each run of 16 keys of the tiles in flight.  Tile t's scores
// are waited for while at most tiles t and t + 1 have left their buffers, so at
// most kKeyTiles more have been asked for.
constexpr int kScaleTiles = 8;
template <bool kF8>
struct TreeSmem : SmemT<kF8> {
  Scan scan;
  TreeSegs segs;
  alignas(16) float ks[kF8 ? kScaleTiles : 1][kBN / 16];
  float qs[kF8 ? TreeSegs::kDepth : 1][2][kF8 ? kBM : 1];  // scales of a segment's query rows, by its slot and stream
};
template <bool kF8>
constexpr size_t kTreeSmemBytes = sizeof(TreeSmem<kF8>) + 1024;
static_assert(kTreeSmemBytes<false> <= 232448 && kTreeSmemBytes<true> <= 232448, "shared memory budget");
static_assert(kScaleTiles >= SmemT<true>::kKeyTiles + 2, "scales of the tiles in flight");

// The producer warp of K or of V: a tile's codes, one copy per page (lanes 0-7),
// into the second half of the tile's buffer.  (Copies are what a producer has
// too little time for: with the scales copied too, in pieces of 32, the kernel
// took half as long again.)
template <class S, int kDepth>
__device__ __forceinline__ void produce(const TreeArgs &a, S &sm, uint8_t (&ring)[kDepth][kTileBytes],
                                        uint64_t (&load)[kDepth], uint64_t (&free)[kDepth], const int8_t *code_base,
                                        const WaitCtx &w) {
  const int lane = threadIdx.x & 31, ps = a.p.page_size;
  const int at = lane * ps;  // the lane's first row in the tile
  int issued[kDepth] = {};
  Ring<kDepth> r;
  TreeReader sr;
  bool ok = true;
  while (ok && (ok = sr.get(sm.segs, w))) {
    const Seg &s = sr.seg(sm.segs);
    const int n = s.n, t0 = s.t0, head = s.head;
    const int64_t table = s.k_base;
    const int32_t keys = static_cast<int32_t>(s.keys);
    sr.done(sm.segs);
    if (n == 0) break;
    // the page of this lane in a tile, read one tile ahead
    auto page_of = [&](int t) {
      const int32_t p0 = (t0 + t) * kBN + at;
      return at < kBN && t < n && p0 < keys ? page_at(a, table, p0) : 0;
    };
    int32_t page = page_of(0);
    for (int t = 0; t < n; ++t) {
      const int32_t left = keys - (t0 + t) * kBN, valid = left < kBN ? left : kBN;
      const int64_t src = (static_cast<int64_t>(page) * a.p.kv_heads + head) << a.p.page_shift;
      page = page_of(t + 1);
      if (!(ok = warp_wait(smem_u32(&free[r.slot]), r.phase ^ 1u, w))) break;
      const uint32_t bar = smem_u32(&load[r.slot]);
      if (lane == 0) mbar_arrive_expect_tx(bar, valid * 128);
      __syncwarp();
      if (at < valid)
        bulk_g2s(smem_u32(ring[r.slot]) + kChunkBytes + at * 128, code_base + src * 128,
                 (valid - at < ps ? valid - at : ps) * 128, bar);
      ++issued[r.slot];
      r.next();
    }
  }
  // every copy that was issued must land before the CTA exits, also where
  // another warp gives up behind the last of them
  for (int x = 0; x < kDepth; ++x)
    if (issued[x]) mbar_wait_drain(smem_u32(&load[x]), (issued[x] - 1) & 1, kDrainNs);
}

// e4m3: the producer warp of K.  Whole pages by TMA with the 128-byte swizzle
// (what lies behind the sequence is masked in the scores), and for each run of 16
// keys what its scores are multiplied with: fp16(scale) times softmax_scale in log2
// units; behind the sequence 1.  At least 2^-60: times a query row's factor, at least
// 2^-66 (split_row), it is no less than fp32's least normal number, so that a masked
// score stays -infinity and is never -infinity times 0.  A factor below that belongs
// to scores that do not count: 128 products of a code (at most 448) and a query
// element (at most 65504, 2^16) come to less than 2^32, times 2^-60 to 2^-28 in log2 units.
__device__ __forceinline__ void produce_keys(const TreeArgs &a, TreeSmem<true> &sm, const CUtensorMap *map,
                                             const WaitCtx &w) {
  constexpr int kDepth = SmemT<true>::kKeyTiles;
  const int lane = threadIdx.x & 31, ps = a.p.page_size;
  const int at = lane * ps, at16 = lane * 16;  // the lane's first row in the tile: of its page, of its run
  int issued[kDepth] = {};
  Ring<kDepth> r;
  TreeReader sr;
  uint32_t tile = 0;
  bool ok = true;
  if (lane == 0) prefetch_tmap(map);
  while (ok && (ok = sr.get(sm.segs, w))) {
    const Seg &s = sr.seg(sm.segs);
    const int n = s.n, t0 = s.t0, head = s.head;
    const int64_t table = s.k_base;
    const int32_t keys = static_cast<int32_t>(s.keys);
    sr.done(sm.segs);
    if (n == 0) break;
    // the pages of this lane in a tile, read one tile ahead
    auto page_of = [&](int t, int row) {
      const int32_t p0 = (t0 + t) * kBN + row;
      return row < kBN && t < n && p0 < keys ? page_at(a, table, p0) : 0;
    };
    auto scale_of = [&](int t, int32_t pg) {
      const bool in = at16 < kBN && t < n && (t0 + t) * kBN + at16 < keys;
      return in ? __ldg(a.k_page_scales + static_cast<int64_t>(pg) * a.p.kv_heads + head) : 0.f;
    };
    int32_t page = page_of(0, at), page16 = page_of(0, at16);
    float scale = scale_of(0, page16);
    page16 = page_of(1, at16);
    for (int t = 0; t < n; ++t, ++tile) {
      const int32_t left = keys - (t0 + t) * kBN, valid = left < kBN ? left : kBN;
      const int32_t row = (page * a.p.kv_heads + head) << a.p.page_shift;
      page = page_of(t + 1, at);
      if (!(ok = warp_wait(smem_u32(&sm.k_free[r.slot]), r.phase ^ 1u, w))) break;
      const uint32_t bar = smem_u32(&sm.k_load[r.slot]);
      if (lane == 0) mbar_arrive_expect_tx(bar, (((valid + ps - 1) >> a.p.page_shift) << a.p.page_shift) * 128);
      __syncwarp();
      if (at < valid) tma_load_2d(smem_u32(sm.k[r.slot]) + at * 128, map, 0, row, bar);
      if (at16 < kBN) {
        float f = __half2float(__float2half_rn(scale)) * a.scale_log2;
        asm("max.NaN.f32 %0, %0, 0f21800000;" : "+f"(f));  // at least 2^-60; NaN stays
        sm.ks[tile % kScaleTiles][lane] = at16 < valid ? f : 1.f;
        mbar_arrive(bar);
      }
      scale = scale_of(t + 1, page16);
      page16 = page_of(t + 2, at16);
      ++issued[r.slot];
      r.next();
    }
  }
  for (int x = 0; x < kDepth; ++x)
    if (issued[x]) mbar_wait_drain(smem_u32(&sm.k_load[x]), (issued[x] - 1) & 1, kDrainNs);
}

// e4m3: a row's lane (values 8l .. 8l+7 and 64 + 8l ..) as the sum of two e4m3 parts
// times a power of two that all its lanes share, with which the row's largest lies in
// (224, 448]: the first part leaves at most 4 bits of a bf16 value's 8, which the second
// holds exactly where they reach down to its least step, 2^-9: for values from 2^-2 on,
// 2^-9 of the largest or less.  Below, it is off by half that step, 2^-17 of the largest.  The power is 2^-66 or
// more (see produce_keys), so a row whose largest element is below 224 2^-66 holds its
// elements to 2^-76.
__device__ __forceinline__ float split_row(const float (&v)[16], uint2 (&hi)[2], uint2 (&lo)[2]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  // least e with top <= 448 2^e, at least -66, and kept where 2^-e is an fp32 number
  const uint32_t u = __float_as_uint(top);
  const int e = min(max(static_cast<int>(u >> 23) - 135 + ((u & 0x7FFFFFu) > 0x600000u), -66), 120);
  const float m = __int_as_float((127 - e) << 23);
  uint32_t c[2][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x0 = v[4 * k] * m, x1 = v[4 * k + 1] * m, x2 = v[4 * k + 2] * m, x3 = v[4 * k + 3] * m;
    c[0][k] = pack_e4m3x4(x0, x1, x2, x3);
    const uint32_t a = e4m3x2_to_f16x2(c[0][k] & 0xFFFFu), b = e4m3x2_to_f16x2(c[0][k] >> 16);
    const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    c[1][k] = pack_e4m3x4(x0 - fa.x, x1 - fa.y, x2 - fb.x, x3 - fb.y);
  }
  hi[0] = make_uint2(c[0][0], c[0][1]);
  hi[1] = make_uint2(c[0][2], c[0][3]);
  lo[0] = make_uint2(c[1][0], c[1][1]);
  lo[1] = make_uint2(c[1][2], c[1][3]);
  return __int_as_float((127 + e) << 23);
}

// Query rows of a segment, from row w0 on and every kStep rows four of them, come into
// rows t0 .. of the swizzled K-major tile in two steps: copied as they are (load_rows, a
// group of asynchronous copies), then, by the same lanes and in the same places,
// rotated: q' = fp16(q H); e4m3: the two parts of q, each a tile of half the size, and
// the rows' scales to `scales`.  Zeros behind the segment's rows, up to the end of a
// softmax warp's 32.  8 lanes hold a row (values 8l .. 8l+7 and 64 + 8l .. of it).
// Four warps take 4 rows each in turn (kStep 16), so that few rows are shared evenly
// (e4m3 drafts 52.7 -> 50.7 us), or 32 rows each (4), which full tiles do as well with.
// Loops that are not unrolled: instructions that run once a segment are waited for
// (unrolled, this took 10 us; e4m3, 8 rows at a time, 4 lanes each, 230 instructions for
// 150: drafts 53.4 for 52.5 us).  A segment's first scores wait for this: stream 1's
// rows are asked for before stream 0's are rotated (e4m3, 16384 tokens 428 -> 423 us,
// chunks 161 -> 158).
template <bool kF8, int kStep>
__device__ __forceinline__ void load_rows(const TreeArgs &a, const Seg &s, uint8_t *tile, int w0, int t0) {
  const int lane = threadIdx.x & 31, l = lane & 7, ti = t0 + (lane >> 3);
  if (kStep == 16 || w0 < s.rows) {
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
      const int row = w0 + it * kStep + (lane >> 3);
      const bool in = row < s.rows;
      if (kStep == 16 && w0 - t0 + ((t0 + it * kStep) & ~31) >= s.rows) break;
      const int x = s.row0 + (in ? row : 0), node = node_of<kF8>(a, x), h = s.head * a.group + (x - node * a.group);
      const uint16_t *src = a.q.data + h * a.q.head_stride + (s.q_base + node) * a.q.row_stride + 8 * l;
      const uint32_t dst = smem_u32(tile) + sw128_off(ti + kStep * it, l);
      copy16_async(dst, src, in);
      copy16_async(dst + kChunkBytes, src + 64, in);
    }
  }
  copy16_commit();
}
template <bool kF8, int kStep>
__device__ __forceinline__ void rotate_rows(int rows, uint8_t *tile, float *scales, int w0, int t0) {
  const int lane = threadIdx.x & 31, l = lane & 7, ti = t0 + (lane >> 3);
  if (w0 < rows) {
#pragma unroll 1
    for (int it = 0; it < 8 && w0 + it * kStep < rows; ++it) {
      uint4 *lo = reinterpret_cast<uint4 *>(tile + sw128_off(ti + kStep * it, l));
      uint4 *hi = reinterpret_cast<uint4 *>(tile + kChunkBytes + sw128_off(ti + kStep * it, l));
      float v[16];
      unpack_bf16x8(*lo, v);
      unpack_bf16x8(*hi, v + 8);
      if constexpr (kF8) {
        uint2 c[2][2];
        const float scale = split_row(v, c[0], c[1]);
        if (l == 0) scales[ti + kStep * it] = scale;
        __syncwarp();  // (a row's parts lie over its values)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint8_t *to = tile + p * kChunkBytes + (l & 1) * 8;
          *reinterpret_cast<uint2 *>(to + sw128_off(ti + kStep * it, l >> 1)) = c[p][0];
          *reinterpret_cast<uint2 *>(to + sw128_off(ti + kStep * it, 4 + (l >> 1))) = c[p][1];
        }
        continue;
      }
      fwht128_oct(v, l);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= kInvSqrt128;
      *lo = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                       pack_f16x2(v[6], v[7]));
      *hi = make_uint4(pack_f16x2(v[8], v[9]), pack_f16x2(v[10], v[11]), pack_f16x2(v[12], v[13]),
                       pack_f16x2(v[14], v[15]));
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// e4m3, values only: dequant_tile for a warp's 32 rows, which have two scales (one for each
// run of 16 keys); zeros in the rows from `left` on, whose codes may be anything,
// NaN among them.
__device__ __forceinline__ void dequant_tile_e4m3(uint8_t *tile, const uint32_t (&scale)[2], int32_t left,
                                                  const attn::DqOffsets &off) {
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    uint4 raw = *reinterpret_cast<const uint4 *>(tile + off.ld8 + it * 512);
    if (4 * it >= left) raw = make_uint4(0, 0, 0, 0);
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const __half2 s = *reinterpret_cast<const __half2 *>(&scale[it >> 2]);
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t f = e4m3x2_to_f16x2(k & 1 ? in[k >> 1] >> 16 : in[k >> 1] & 0xFFFFu);
      const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&f), s);
      o[k] = *reinterpret_cast<const uint32_t *>(&v);
    }
    uint8_t *row = tile + it * 512;
    *reinterpret_cast<uint4 *>(row + off.st[it & 1][0]) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4 *>(row + off.st[it & 1][1]) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// e4m3: scores times their factors, less `ref`, in TMEM: shift_tile.  The product is
// rounded as the maximum's is: its own score less itself has to be 0.
__device__ __forceinline__ void shift_tile_e4m3(uint32_t tS, float ref, float qs, const float *ks) {
#pragma unroll 1
  for (int g = 0; g < 8; ++g) {
    const float m = qs * ks[g];
    uint32_t x[16];
    tmem_ld16(tS + 16 * g, x);
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[c]), m), ref));
    tmem_st16(tS + 16 * g, x);
  }
  tmem_wait_st();
}

// e4m3: softmax_tile with scores in log2 units, which the running maximum is in too:
// those of a run of 16 keys times qs (the row's scale) and ks (of the keys), another
// factor in the same instructions.  `half` is told of the first 64 keys' weights.  Runs
// share their scale two by two but for pages of 16, so that the loads' maxima of 32
// columns serve.
__device__ __forceinline__ void softmax_tile_e4m3(uint32_t tS, uint32_t tO, bool first, float qs, const float *ks,
                                                  bool pages16, uint32_t half, Row &r) {
  float s[128];
  float m4[4];
  const float4 k0 = reinterpret_cast<const float4 *>(ks)[0], k1 = reinterpret_cast<const float4 *>(ks)[1];
  float f[8] = {k0.x * qs, k0.y * qs, k0.z * qs, k0.w * qs, k1.x * qs, k1.y * qs, k1.z * qs, k1.w * qs};
  tmem_ld128_max(tS, *reinterpret_cast<uint32_t(*)[128]>(s), m4);
  float mt;
  if (!pages16) {
    mt = fmax3(m4[0] * f[0], m4[1] * f[2], fmaxf(m4[2] * f[4], m4[3] * f[6]));
  } else {
    mt = -INFINITY;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float x = s[16 * g];
#pragma unroll
      for (int c = 1; c < 15; c += 2) x = fmax3(x, s[16 * g + c], s[16 * g + c + 1]);
      mt = fmaxf(mt, fmaxf(x, s[16 * g + 15]) * f[g]);
    }
  }
  if (first) {
    r.m = mt;
    r.l = 0.f;
  }
  const bool need = mt - r.m > kLazyRescaleLog2, far = fabsf(mt) > kFusedMaxLog2 && mt != kNoMax;
  bool shifted = false;
  if (__any_sync(0xffffffffu, need || far)) {
    if (!first) {
      const float alpha = need ? ex2(r.m - mt) : 1.f;
      if (need) {
        r.l *= alpha;
        r.m = mt;
      }
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(tO + c * 16, o);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        tmem_st16(tO + c * 16, o);
      }
    }
    if (__any_sync(0xffffffffu, far)) {
      shift_tile_e4m3(tS, r.m == kNoMax ? 0.f : r.m, qs, ks);
      tmem_ld128_max(tS, *reinterpret_cast<uint32_t(*)[128]>(s), m4);
#pragma unroll
      for (int g = 0; g < 8; ++g) f[g] = 1.f;
      shifted = true;
    }
  }
  const float bias = r.m == kNoMax || shifted ? kWeightLog2 : kWeightLog2 - r.m;  // (kNoMax: all scores are -infinity)
  const float2 nm = make_float2(bias, bias);
  float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int c = h * 64 + 2 * k;
      float2 e = __ffma2_rn(make_float2(s[c], s[c + 1]), make_float2(f[c >> 4], f[c >> 4]), nm);
      e.x = ex2(e.x);
      e.y = ex2(e.y);
      if (k & 1) acc1 = __fadd2_rn(acc1, e);
      else acc0 = __fadd2_rn(acc0, e);
      pk[k] = attn::pack2<true>(e.x, e.y);
    }
    tmem_st32(tS + h * 32, pk);
    if (h == 0) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(half);
    }
  }
  tmem_wait_st();
  const float2 acc = __fadd2_rn(acc0, acc1);
  r.l += acc.x + acc.y;
}

// The same in a loop over 32 columns, which are loaded again: a quarter of the code.
// Where few warps have rows, instructions are what a tile waits for (1.4 cycles an
// issue, 0.3 with 256 rows): 24 x 8192 rows with 5 drafted tokens 58.8 -> 54.2 us, 64
// rows of 128 x 1024 144 -> 131; 256 rows, 16384 of them: 425 -> 459.
__device__ __forceinline__ void softmax_tile_e4m3_rolled(uint32_t tS, uint32_t tO, bool first, float qs, const float *ks,
                                                  bool pages16, uint32_t half, Row &r) {
  float mt;
  {
    float s[128], m4[4];
    tmem_ld128_max(tS, *reinterpret_cast<uint32_t(*)[128]>(s), m4);
    if (!pages16) {
      mt = fmax3(m4[0] * ks[0], m4[1] * ks[2], fmaxf(m4[2] * ks[4], m4[3] * ks[6])) * qs;
    } else {
      mt = -INFINITY;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float x = s[16 * g];
#pragma unroll
        for (int c = 1; c < 15; c += 2) x = fmax3(x, s[16 * g + c], s[16 * g + c + 1]);
        mt = fmaxf(mt, fmaxf(x, s[16 * g + 15]) * ks[g]);
      }
      mt *= qs;
    }
  }
  if (first) {
    r.m = mt;
    r.l = 0.f;
  }
  const bool need = mt - r.m > kLazyRescaleLog2, far = fabsf(mt) > kFusedMaxLog2 && mt != kNoMax;
  bool shifted = false;
  if (__any_sync(0xffffffffu, need || far)) {
    if (!first) {
      const float alpha = need ? ex2(r.m - mt) : 1.f;
      if (need) {
        r.l *= alpha;
        r.m = mt;
      }
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(tO + c * 16, o);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        tmem_st16(tO + c * 16, o);
      }
    }
    if (__any_sync(0xffffffffu, far)) {
      shift_tile_e4m3(tS, r.m == kNoMax ? 0.f : r.m, qs, ks);
      shifted = true;
    }
  }
  const float bias = r.m == kNoMax || shifted ? kWeightLog2 : kWeightLog2 - r.m;  // (kNoMax: all scores are -infinity)
  const float2 nm = make_float2(bias, bias);
  float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    float s[32];
    tmem_ld32(tS + 32 * g, *reinterpret_cast<uint32_t(*)[32]>(s));
    const float f0 = shifted ? 1.f : ks[2 * g] * qs, f1 = shifted ? 1.f : ks[2 * g + 1] * qs;
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float f = k < 8 ? f0 : f1;
      float2 e = __ffma2_rn(make_float2(s[2 * k], s[2 * k + 1]), make_float2(f, f), nm);
      e.x = ex2(e.x);
      e.y = ex2(e.y);
      if (k & 1) acc1 = __fadd2_rn(acc1, e);
      else acc0 = __fadd2_rn(acc0, e);
      pk[k] = attn::pack2<true>(e.x, e.y);
    }
    tmem_st16(tS + 16 * g, pk);
    if (g == 1) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(half);
    }
  }
  tmem_wait_st();
  const float2 acc = __fadd2_rn(acc0, acc1);
  r.l += acc.x + acc.y;
}

// kRolled (e4m3): for a mean of up to 128 rows.
template <bool kF8, bool kWide, bool kRolled>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_k, const TreeArgs a) {
  // query rows: 4 for each of four warps in turn, or 32 (see load_rows)
  constexpr int kStep = !kF8 || kRolled ? 16 : 4, kEach = kStep == 16 ? 4 : 32;
  extern __shared__ uint8_t smem_raw[];
  TreeSmem<kF8> &sm = *reinterpret_cast<TreeSmem<kF8> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Workspace ws = workspace_of<kF8>(a);

  // the join may start its CTAs; it waits there until this grid is done
  if (tid == 0) pdl_launch_dependents();
  find_run<kF8 ? kE4m3Many : kKvi8r, kThreads>(a, sm.scan, reinterpret_cast<int64_t *>(sm.q[0]));
  if (sm.scan.u0 >= sm.scan.u1) {
    if (tid == 0) ws.split[blockIdx.x].parts = 0;
    return;
  }

  if (tid == 0) {
    init_seg_ring(sm.segs, 15);
    init_barriers<kF8>(sm, true);
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const WaitCtx w{a.p.err, &sm.abort, a.timeout_ns};
  TreeReader sr;

  if (warp < 8) {
    // =================================================== softmax warpgroups
    reg_alloc<kRegSoftmax>();
    const int q = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + q * 128, tO = tmem + lane_base + 256 + q * 128;
    const float c2 = kF8 ? 1.f : a.scale_log2;  // (e4m3: maxima are in log2 units)
    const int i = tid & 127;
    uint32_t s_phase = 0;
    bool first = true;
    uint32_t tile0 = 0;  // e4m3: tiles of the segments before
    StreamEnd fin;
    while (sr.get(sm.segs, w)) {
      const Seg &s = sr.seg(sm.segs);
      if (s.n == 0) break;
      const int base_row = s.two ? q * kBM : 0;
      const int r = base_row + i;
      const int w0 = base_row + (warp & 3) * 32;  // the warp's first row
      const bool warp_on = w0 < s.rows;
      if (first) {
        // nobody is busy yet: every warp rotates its own rows
        first = false;
        if (has_tiles(s, q)) {
          const int t0 = (warp & 3) * kEach;
          load_rows<kF8, kStep>(a, s, sm.q[q], base_row + t0, t0);
          copy16_wait();
          rotate_rows<kF8, kStep>(s.rows, sm.q[q], sm.qs[kF8 ? sr.r.slot : 0][q], base_row + t0, t0);
          if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
        }
      }
      const int32_t base_key = static_cast<int32_t>(s.keys) - s.nodes, pos0 = s.t0 * kBN;
      uint64_t path = 0;
      int32_t sees = 0, warp_sees = 0;  // e4m3: keys that the row, and all the warp's rows, see
      if constexpr (kF8) {
        sees = keys_seen(a, s, s.row0 + (r < s.rows ? r : s.rows - 1));
        warp_sees = keys_seen(a, s, s.row0 + w0);
      } else {
        if (r < s.rows) path = path_of(a, s.q_base, node_of<kF8>(a, s.row0 + r));
      }
      Row row{kNoMax, 0.f};
      bool ok = true;
      const int step = tile_step(s), end = end_tile(s, q), t_first = first_tile(s, q);
      for (int t = t_first; t < end; t += step) {
        if (!warp_wait(smem_u32(&sm.s_full[q]), s_phase, w)) {
          ok = false;
          break;
        }
        s_phase ^= 1u;
        tc_fence_after();
        if (warp_on) {
          const int32_t pos = pos0 + t * kBN;
          uint32_t see[4];
          if constexpr (kF8) {
            if (pos + kBN > warp_sees) {
              prefix_mask(sees - pos, see);
              mask_tile(tS, see);
            }
          } else if (pos + kBN > base_key) {
            tree_mask(pos, base_key, path, see);
            mask_tile(tS, see);
          }
          if constexpr (kF8) {
            const float qs = sm.qs[sr.r.slot][q][i], *ks = sm.ks[(tile0 + t) % kScaleTiles];
            const bool pages16 = a.p.page_size == 16;
            if constexpr (!kRolled)
              softmax_tile_e4m3(tS, tO, t == t_first, qs, ks, pages16, smem_u32(&sm.p_half[q]), row);
            else
              softmax_tile_e4m3_rolled(tS, tO, t == t_first, qs, ks, pages16, smem_u32(&sm.p_half[q]), row);
          } else {
            softmax_tile<true>(tS, tO, t == t_first, c2, row);
          }
        } else if (kF8 && lane == 0) {
          mbar_arrive(smem_u32(&sm.p_half[q]));
        }
        tc_fence_before();
        __syncwarp();
        // (a diagnostic may withhold one tile's arrival: see withhold_p_tile1)
        if (lane == 0 && t + 1 != a.withhold_p_tile1) mbar_arrive(smem_u32(&sm.p_full[q]));
      }
      bool joined;
      float ga, gb;
      const End e = ok ? fin.at_end(sm, s, q, warp_on, row, c2, &joined, &ga, &gb, w) : kFailed;
      if (e == kFailed) break;
      if (e == kWrite) {
        // (without the weights' factor)
        row.l *= kWeightInv;
        ga *= kWeightInv;
        gb *= kWeightInv;
        const bool live = r < s.rows;
        if (kF8 && s.whole) {
          const float inv = 1.f / row.l, gx = ga * inv, gy = gb * inv;
          const int x = s.row0 + (live ? r : 0), node = node_of<kF8>(a, x), h = s.head * a.group + (x - node * a.group);
          uint16_t *dst = a.o.data + h * a.o.head_stride + (s.q_base + node) * a.o.row_stride;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(tO + c * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= gx;
            if (joined) {
              float y[32];
              tmem_ld32(tO + 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(y));
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = fmaf(y[k], gy, o[k]);
            }
            if (live) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                uint32_t w8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w8[k] = pack_bf16x2(o[16 * g + 2 * k], o[16 * g + 2 * k + 1]);
                uint16_t *to = dst + 32 * c + 16 * g;
                if constexpr (kWide) {
                  st_global_v8(to, w8);
                } else {
                  reinterpret_cast<uint4 *>(to)[0] = make_uint4(w8[0], w8[1], w8[2], w8[3]);
                  reinterpret_cast<uint4 *>(to)[1] = make_uint4(w8[4], w8[5], w8[6], w8[7]);
                }
              }
            }
          }
          if (live && a.lse) a.lse[h * a.nodes + s.q_base + node] = kLn2 * (row.m * c2 + log2f(row.l));
        } else if (s.whole) {
          // H128 = [[H64, H64], [H64, -H64]]: the output's halves are the
          // transforms of the sum and of the difference of O's; a loop over
          // them (code of half the size, see mask_tile)
          const float inv = kInvSqrt128 / row.l, gx = ga * inv, gy = gb * inv;
          const int x = s.row0 + r, node = node_of<kF8>(a, live ? x : 0), h = s.head * a.group + (x - node * a.group);
          uint16_t *dst = a.o.data + h * a.o.head_stride + (s.q_base + node) * a.o.row_stride;
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            float o[64];
            const float sx = hf ? -gx : gx, sy = hf ? -gy : gy;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float lo[32], hi[32];
              tmem_ld32(tO + c * 32, *reinterpret_cast<uint32_t(*)[32]>(lo));
              tmem_ld32(tO + 64 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(hi));
#pragma unroll
              for (int k = 0; k < 32; ++k) o[32 * c + k] = fmaf(hi[k], sx, lo[k] * gx);
            }
            if (joined) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float lo[16], hi[16];
                tmem_ld16(tO + 128 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(lo));
                tmem_ld16(tO + 192 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(hi));
#pragma unroll
                for (int k = 0; k < 16; ++k) o[16 * c + k] += fmaf(hi[k], sy, lo[k] * gy);
              }
            }
            fwht64_packed(o);
            if (live) {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint32_t c[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) c[k] = pack_bf16x2(o[16 * g + 2 * k], o[16 * g + 2 * k + 1]);
                uint16_t *to = dst + 64 * hf + 16 * g;
                if constexpr (kWide) {
                  st_global_v8(to, c);
                } else {
                  reinterpret_cast<uint4 *>(to)[0] = make_uint4(c[0], c[1], c[2], c[3]);
                  reinterpret_cast<uint4 *>(to)[1] = make_uint4(c[4], c[5], c[6], c[7]);
                }
              }
            }
          }
          if (live && a.lse) a.lse[h * a.nodes + s.q_base + node] = kLn2 * (row.m * c2 + log2f(row.l));
        } else {
          const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + (s.t0 > 0 ? 0 : 1)) * ws.rows + r;
          float *dst = ws.o + at * 128;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float x[16];
            tmem_ld16(tO + c * 16, *reinterpret_cast<uint32_t(*)[16]>(x));
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] *= ga;
            if (joined) {
              float y[16];
              tmem_ld16(tO + 128 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(y));
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = fmaf(y[k], gb, x[k]);
            }
            if (live) {
              st_global_v8(dst + 16 * c, *reinterpret_cast<const uint32_t(*)[8]>(x));
              st_global_v8(dst + 16 * c + 8, *reinterpret_cast<const uint32_t(*)[8]>(x + 8));
            }
          }
          if (live) ws.ml[at] = make_float2(row.m, row.l);
        }
      }
      fin.read_done(sm, joined);
      tile0 += s.n;
      sr.done(sm.segs);
    }
  } else if (warp < 12) {
    // ======================================================= dequantisers
    reg_dealloc<kRegDequant>();
    const int dw = warp - 8;
    const attn::DqOffsets off = attn::dq_offsets(dw, lane);
    const int rr = 2 * (lane >> 4) + ((lane >> 2) & 1);
    Ring<SmemT<kF8>::kKeyTiles> kr;
    Ring<SmemT<kF8>::kValueTiles> vr;
    auto dequant = [&](uint8_t *tile, const uint16_t (&sc)[8]) {
      attn::dequant_tile(tile, sc, off);
      fence_proxy_async_smem();
      __syncwarp();
    };
    uint32_t q_phase[2] = {0, 0};
    bool ok = true, first = true;
    while (ok && (ok = sr.get(sm.segs, w))) {
      const Seg &s = sr.seg(sm.segs);
      const int n = s.n, head = s.head;
      const int64_t table = s.k_base;
      const int32_t keys = static_cast<int32_t>(s.keys);
      int32_t pos = s.t0 * kBN + dw * 32;  // the warp's first row
      if (n == 0) break;
      // the query rows of every segment but the first (see rotate_rows): the
      // softmax warps are then still at the output of the one before
      for (int q = 0; q < 2; ++q) {
        if (!has_tiles(s, q)) continue;
        q_phase[q] ^= 1u;
        if (first) continue;
        if (!(ok = warp_wait(smem_u32(&sm.q_free[q]), q_phase[q], w))) break;
        load_rows<kF8, kStep>(a, s, sm.q[q], (s.two ? q * kBM : 0) + dw * kEach, dw * kEach);
      }
      // (stream 1's rows come while stream 0's are rotated.  kvi8r: unrolled, with which 64
      // nodes of 32 heads over 8 take 228 us on 2 x 131072 rows and 315 on 128 x 2048; 242 and
      // 335 as a loop, where the compiler spills more.  e4m3: 64 rows over 128 x 1024 120 us
      // as a loop, 127 unrolled.)
#pragma unroll(kF8 ? 1 : 2)
      for (int q = 0; q < 2; ++q) {
        if (first || !ok || !has_tiles(s, q)) continue;
        if (q == 0 && has_tiles(s, 1)) copy16_wait_but<1>();
        else copy16_wait();
        rotate_rows<kF8, kStep>(s.rows, sm.q[q], sm.qs[kF8 ? sr.r.slot : 0][q], (s.two ? q * kBM : 0) + dw * kEach,
                                dw * kEach);
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
      }
      copy16_wait();  // (also where a wait for the second has run out)
      first = false;
      sr.done(sm.segs);
      if (!ok) break;
      // the pages of its rows 0-15 and 16-31, read one tile ahead
      const int ps = a.p.page_size;
      auto pages_of = [&](int32_t p, int32_t (&pg)[2]) {
        pg[0] = p < keys ? page_at(a, table, p) : 0;
        pg[1] = ps == 16 ? (p + 16 < keys ? page_at(a, table, p + 16) : 0) : pg[0];
      };
      int32_t pg[2];
      pages_of(pos, pg);
      for (int t = 0; t < n; ++t, pos += kBN) {
        if constexpr (kF8) {
          // V's scales of the warp's two runs of 16 keys, read before the wait
          uint32_t sv[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int64_t at = static_cast<int64_t>(pg[hf]) * a.p.kv_heads + head;
            // (behind the sequence 0: page 0, which stands for one there, may hold NaN)
            const float f = pos + 16 * hf < keys ? __ldcg(a.v_page_scales + at) : 0.f;
            sv[hf] = pack_f16x2(f, f);
          }
          const int32_t left = keys - pos - rr;
          if (t + 1 < n) pages_of(pos + kBN, pg);
          if (!(ok = warp_wait(smem_u32(&sm.v_load[vr.slot]), vr.phase, w))) break;
          dequant_tile_e4m3(sm.v[vr.slot], sv, left, off);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.v_ready[vr.slot]));
          vr.next();
          continue;
        }
        // the scales of the lane's rows (behind the sequence: 0), read before
        // the waits
        uint16_t sck[8], scv[8];
        const int32_t left = keys - pos - rr;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int64_t src = ((static_cast<int64_t>(pg[hf]) * a.p.kv_heads + head) << a.p.page_shift) +
                              ((pos + 16 * hf) & (ps - 1)) + rr;
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const bool in = 16 * hf + 4 * it < left;
            sck[4 * hf + it] = in ? __ldcg(a.p.k_scales + src + 4 * it) : 0;
            scv[4 * hf + it] = in ? __ldcg(a.p.v_scales + src + 4 * it) : 0;
          }
        }
        if (t + 1 < n) pages_of(pos + kBN, pg);
        if (!(ok = warp_wait(smem_u32(&sm.k_load[kr.slot]), kr.phase, w))) break;
        dequant(sm.k[kr.slot], sck);
        if (lane == 0) mbar_arrive(smem_u32(&sm.k_ready[kr.slot]));
        kr.next();
        if (!(ok = warp_wait(smem_u32(&sm.v_load[vr.slot]), vr.phase, w))) break;
        dequant(sm.v[vr.slot], scv);
        if (lane == 0) mbar_arrive(smem_u32(&sm.v_ready[vr.slot]));
        vr.next();
      }
    }
  } else {
    reg_dealloc<kRegIssue>();
    if (warp == 12) {
      if constexpr (kF8) produce_keys(a, sm, &tm_k, w);
      else produce(a, sm, sm.k, sm.k_load, sm.k_free, a.p.k_codes, w);
    } else if (warp == 14) {
      produce(a, sm, sm.v, sm.v_load, sm.v_free, a.p.v_codes, w);
    } else if (warp == 13) {
      MmaState<kF8> m;
      mma_setup<kF8>(m, sm, false);
      while (sr.get(sm.segs, w)) {
        const Seg s = sr.seg(sm.segs);
        sr.done(sm.segs);
        if (s.n == 0 || !mma_segment<true, kF8>(m, sm, s, false, w)) break;
      }
      // every MMA issued must finish before TMEM is released
      mma_commit(m.go, smem_u32(&sm.drain));
      mbar_wait_drain(smem_u32(&sm.drain), 0, kDrainNs);
    } else if (warp == 15) {
      publish_segments<kF8 ? kE4m3Many : kKvi8r>(a, sm.scan, ws, sm.segs, w, [](const Seg &, int) { return true; });
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the items that lie on several CTAs: block column b takes the one that
// CTA b + 1 is the second of.  A warp takes 4 rows, 8 lanes each, in the order
// of fwht128_oct; where an item has fewer rows than the block's warps hold, the
// warps share its parts (warp w of `ways` takes parts w, w + ways, ..) and meet
// in shared memory.  Parts are added in a fixed order.
constexpr int kJoinRows = 4, kJoinWarpsFew = 16, kJoinWarpsMany = 4;
template <bool kF8>
__global__ void __launch_bounds__(kJoinWarpsFew * 32) join_kernel(const TreeArgs a) {
  extern __shared__ float4 sh_o[];  // [warps][4][32], if the warps share parts
  __shared__ float2 sh_ml[kJoinWarpsFew][kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x + 1;
  const int l8 = lane & 7, sub = lane >> 3, warps = blockDim.x >> 5;
  // (no thread leaves before this, so the grids end in stream order)
  pdl_wait_prerequisites();
  const Workspace ws = workspace_of<kF8>(a);
  const Split sp = ws.split[b];
  if (sp.parts == 0) return;
  const int lg = ws.rows <= 4 ? 0 : ws.rows <= 8 ? 1 : ws.rows <= 16 || warps == 4 ? 2 : 3, groups = 1 << lg, ways = warps >> lg;
  const int g = warp & (groups - 1), way = warp >> lg;
  const int r = (blockIdx.y * groups + g) * kJoinRows + sub;
  const bool live = r < sp.rows;
  const float c2 = kF8 ? 1.f : a.scale_log2;
  float m = kNoMax, l = 0.f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  auto add = [&](float2 ml, const float (&p)[16]) {
    const float mn = fmaxf(m, ml.x), ref = mn == kNoMax ? 0.f : mn;
    const float ga = ex2((m - ref) * c2), gb = ex2((ml.x - ref) * c2);
    l = fmaf(l, ga, ml.y * gb);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = fmaf(o[e], ga, p[e] * gb);
    m = mn;
  };
  if (live) {
#pragma unroll 2
    for (int k = way; k < sp.parts; k += ways) {
      const int64_t at = (static_cast<int64_t>(b - 1 + k) * 2 + (k == 0 ? 1 : 0)) * ws.rows + r;
      const float4 *src = reinterpret_cast<const float4 *>(ws.o + at * 128) + 2 * l8;
      const float2 ml = ws.ml[at];
      float p[16];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 f = src[(x >> 1) * 16 + (x & 1)];
        p[4 * x] = f.x;
        p[4 * x + 1] = f.y;
        p[4 * x + 2] = f.z;
        p[4 * x + 3] = f.w;
      }
      add(ml, p);
    }
  }
  if (ways > 1) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      sh_o[(warp * 4 + x) * 32 + lane] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
    if (l8 == 0) sh_ml[warp][sub] = make_float2(m, l);
    __syncthreads();
    if (way > 0) return;
    for (int y = 1; y < ways; ++y) {
      const int from = y * groups + g;
      float p[16];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 f = sh_o[(from * 4 + x) * 32 + lane];
        p[4 * x] = f.x;
        p[4 * x + 1] = f.y;
        p[4 * x + 2] = f.z;
        p[4 * x + 3] = f.w;
      }
      add(sh_ml[from][sub], p);
    }
  }
  if constexpr (!kF8) fwht128_oct(o, l8);
  if (!live) return;
  const float inv = (kF8 ? 1.f : kInvSqrt128) / l;
  const int x = sp.row0 + r, node = node_of<kF8>(a, x), h = sp.head * a.group + (x - node * a.group);
  const int64_t row = sp.q_base + node;
  uint4 *dst = reinterpret_cast<uint4 *>(a.o.data + h * a.o.head_stride + row * a.o.row_stride) + l8;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = pack_bf16x2(o[8 * hi + 2 * k] * inv, o[8 * hi + 2 * k + 1] * inv);
    dst[8 * hi] = make_uint4(c[0], c[1], c[2], c[3]);
  }
  if (a.lse && l8 == 0) a.lse[h * a.nodes + row] = kLn2 * (m * c2 + log2f(l));
}

// (For the kernel of more rows where the page table's width decides.)
template <bool kF8>
size_t workspace_bytes(int32_t group, int64_t nodes, int32_t seqs) {
  const size_t rows = part_rows<kF8>(group, nodes, item_rows_of<kF8>(group, nodes, seqs, kF8LongSpan));
  return kMaxCtas * (sizeof(Split) + 2 * rows * (128 * sizeof(float) + sizeof(float2)));
}

template <bool kF8>
cudaError_t launch_attention(const TreeArgs &args, cudaStream_t stream) {
  TreeArgs a = args;
  a.ctas = a.ctas < kMaxCtas ? a.ctas : kMaxCtas;
  a.item_rows = item_rows_of<kF8>(a.group, a.nodes, a.seqs, a.max_pages << a.p.page_shift);
  a.item_cost = item_cost_of(a.item_rows);
  a.group_magic = kF8 ? static_cast<uint32_t>(((1ull << 32) + a.group - 1) / a.group)
                      : ((1u << 19) + a.group - 1) / a.group;
  a.tile_nodes = kManyRows / a.group;
  cudaError_t e;
  if (a.item_rows < kManyRows) {
    e = kF8 ? launch_chunk_few(a, stream) : launch_tree_few(a, stream);
  } else {
    // whole 32-byte sectors per store where the output's alignment allows
    const bool wide = ((reinterpret_cast<uintptr_t>(a.o.data) | static_cast<uintptr_t>(a.o.head_stride * 2) |
                        static_cast<uintptr_t>(a.o.row_stride * 2)) &
                       31) == 0;
    const bool rolled = kF8 && a.group * a.nodes <= 128ll * a.seqs;
    auto kernel = rolled ? (wide ? tree_kernel<kF8, true, kF8> : tree_kernel<kF8, false, kF8>)
                         : (wide ? tree_kernel<kF8, true, false> : tree_kernel<kF8, false, false>);
    static std::atomic<uint64_t> allowed[4];
    e = allow_smem(kernel, static_cast<int>(kTreeSmemBytes<kF8>), allowed[2 * rolled + wide]);
    if (e != cudaSuccess) return e;
    CUtensorMap tk = {};  // (kvi8r codes come by untiled copies)
    const int64_t rows = (static_cast<int64_t>(a.p.pages) * a.p.kv_heads) << a.p.page_shift;
    if (kF8 && !encode_codes(&tk, a.p.k_codes, rows, a.p.page_size)) return cudaErrorInvalidValue;
    kernel<<<a.ctas, kThreads, kTreeSmemBytes<kF8>, stream>>>(tk, a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  if (a.ctas < 2) return cudaSuccess;
  const int rows = part_rows<kF8>(a.group, a.nodes, a.item_rows);
  const bool few = rows <= 32;  // (one block an item)
  const int warps = few ? kJoinWarpsFew : kJoinWarpsMany;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas - 1, few ? 1 : (rows + kJoinWarpsMany * kJoinRows - 1) / (kJoinWarpsMany * kJoinRows));
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = few ? warps * kJoinRows * 32 * sizeof(float4) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<kF8>, a);
}

}  // namespace
}  // namespace serve
}  // namespace h3kv
