// attend_tree_few.cu -- attention of drafted tokens over the paged kvi8r cache
// for few rows of a sequence and kv head (items of 8, 16 or 32: single tokens
// with grouped heads, short drafts).
//
// Bound by HBM: 260 bytes of cache per key and kv head, against 4 * 128 FLOP
// for each of at most 32 rows.  The 128-row tiles of tcgen05 would be nearly
// empty and would want K and V as fp16 in shared memory, twice the bytes of
// the codes; here the codes go from shared memory to registers, are
// dequantised there and feed warp-level MMAs (m16n8k16) whose 16 is the key
// (or channel) and whose 8 are the rows:
//   S^T [16 keys, 8 rows]     = K' [16, 128]  q'^T [128, 8]
//   O^T [128 channels, 8 rows] += V'^T [128, 16]  P^T [16, 8]
// P^T comes out of S^T's registers by one 8x8 transpose per 8 keys.  A warp
// takes 16 keys of a 128-key tile with a softmax of its own; the warps' results
// are joined at the segment's end.
//
// 8 such warps; producer warps copy whole pages: codes by TMA with the 128-byte
// swizzle (so that the reads below spread over the banks), scales by bulk
// copies, kStages tiles of 33 KB in flight.  A step's codes are taken into
// registers at once, so that a stage is empty while its products run.  Measured,
// 32 query heads over 8, one token each: 32 x 8192 cached rows 94 us (5.8 TB/s),
// 8 x 32768 92 us (5.9), 256 x 1024 111 us (4.9), 1 x 65536 32 us (4.3), 1 x 1024 9
// us; 5 tokens with 32 heads over 32 on 217088 rows 273 us (6.6 TB/s).  Four tokens
// each of 32 x 8192 124 us, eight 161 us: from 16 rows on the issue of the
// products and of what feeds them bounds it.
#include "tree.cuh"

namespace h3kv {
namespace serve {
namespace {

// Consumer warps and ring stages.
constexpr int kWarps = 8, kProducers = 3, kStages = 5;
constexpr int kFewThreads = (kWarps + kProducers + 1) * 32;
constexpr int kCodeBytes = kBN * 128;      // one tile's codes
constexpr int kPitch = 132;                // floats of a row in the join buffer
constexpr int kQPitch = 136;               // values of a query row: 16 bytes aside, so that 8 rows' reads spread
// "No key yet" in a running maximum, which is in log2 units here: finite, so
// that no difference of two infinities arises, and no score is below it.
constexpr float kNoMaxLog2 = -3.4e38f;

template <int kNT>
struct FewSmem {
  uint8_t k[kStages][kCodeBytes];
  uint8_t v[kStages][kCodeBytes];
  float o[kWarps][8][kPitch];              // the warps' O, 8 rows at a time
  uint16_t ks[kStages][kBN], vs[kStages][kBN];
  uint16_t q[TreeSegs::kDepth][8 * kNT][kQPitch];  // q' of a segment's rows, by its slot
  float m[kWarps][8 * kNT], l[kWarps][8 * kNT];
  uint64_t path[TreeSegs::kDepth][8 * kNT];
  uint64_t full[kStages], empty[kStages], q_full[TreeSegs::kDepth];
  Scan scan;
  TreeSegs segs;
  int abort;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two biased code bytes (c + 128) in the low bytes of the half-words of a word
// whose high bytes are 0x64 are the fp16 pair 1024 + c + 128.
__device__ __forceinline__ uint32_t unbias(uint32_t x) {
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480u), __ushort_as_half(0x6480u));  // 1152
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&x), bias);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t scale2(uint32_t x, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&s));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// q' = fp16(q H) of a row in place, by 8 lanes (l: the lane among them).
__device__ __forceinline__ void rotate_row(uint16_t (&row)[kQPitch], int l) {
  uint4 *dst = reinterpret_cast<uint4 *>(row) + l;
  float v[16];
  unpack_bf16x8(dst[0], v);
  unpack_bf16x8(dst[8], v + 8);
  fwht128_oct(v, l);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] *= kInvSqrt128;
  dst[0] = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
  dst[8] = make_uint4(pack_f16x2(v[8], v[9]), pack_f16x2(v[10], v[11]), pack_f16x2(v[12], v[13]),
                      pack_f16x2(v[14], v[15]));
}

// Items of 32 rows: O of a thread takes 128 registers, so the consumers get 224,
// the query fragments are read again for each tile and V's codes only behind
// K's products; 108 bytes a thread are spilled all the same (24 with items of
// 16).  (In two items of 16 rows, 8 nodes of four heads over 32 x 8192
// rows took 234 us; 161 so.)
constexpr uint32_t kRegConsumer = 224, kRegOther = 56;
static_assert(2 * kRegConsumer + kRegOther == 3 * 168, "register split");

template <int kNT>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  using S = FewSmem<kNT>;
  S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Workspace ws = workspace_of(a);

  // the join may start its CTAs; it waits there until this grid is done
  if (tid == 0) pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), kProducers);
      mbar_init(smem_u32(&sm.empty[s]), 8);
    }
    init_seg_ring(sm.segs, kWarps + kProducers);
    for (int i = 0; i < TreeSegs::kDepth; ++i) mbar_init(smem_u32(&sm.q_full[i]), 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  find_run<kFewThreads>(a, sm.scan, reinterpret_cast<int64_t *>(sm.o));
  if (sm.scan.u0 >= sm.scan.u1) {
    if (tid == 0) ws.split[blockIdx.x].parts = 0;
    return;
  }
  const WaitCtx w{a.p.err, &sm.abort, a.timeout_ns};

  TreeReader sr;

  // The walking warp also fetches the query rows (rows behind them 0) and their
  // paths while the consumers are still at the segment before: 256 sequences of
  // 1024 rows 121 -> 115 us.  Of items of 8 rows it rotates them too, 111 us; of
  // 16 rows it takes too long before the first segment (27.3 us for 4 nodes of 8
  // sequences, against 26.4), so there each consumer rotates four.
  constexpr bool kAhead = kNT == 1, kBig = kNT == 4;
  if (warp >= kWarps) {
    if constexpr (kBig) reg_dealloc<kRegOther>();
    if (warp == kWarps + kProducers) {
      publish_segments(a, sm.scan, ws, sm.segs, w, [&](const Seg &s, int slot) {
        const int l = lane & 7;
#pragma unroll 1
        for (int row = lane >> 3; row < 8 * kNT; row += 4) {
          const bool in = row < s.rows;
          const int x = s.row0 + (in ? row : 0), node = node_of(a, x), h = s.head * a.group + (x - node * a.group);
          const uint16_t *src = a.q.data + h * a.q.head_stride + (s.q_base + node) * a.q.row_stride + 8 * l;
          const uint32_t dst = smem_u32(sm.q[slot][row]) + 16 * l;
          copy16_async(dst, src, in);
          copy16_async(dst + 128, src + 64, in);
          if (l == 0) sm.path[slot][row] = in ? path_of(a, s.q_base, node) : 0;
        }
        copy16_wait();
        if constexpr (kAhead) {
#pragma unroll 1
          for (int row = lane >> 3; row < 8 * kNT; row += 4) rotate_row(sm.q[slot][row], l);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[slot]));
        return true;
      });
      return;
    }
    // =========================================================== producers
    // one warp each for K's codes, V's codes and the scales (one warp for all
    // of them was what bounded the kernel); lanes 0-7 take the pages of a
    // tile, lanes 8-15 V's scales
    const int kind = warp - kWarps, ps = a.p.page_size;
    const int at = (lane & 7) * ps;  // the lane's first row in the tile
    const bool lane_on = lane < (kind == 2 ? 16 : 8) && at < kBN;
    const CUtensorMap *map = kind == 0 ? &tm_k : &tm_v;
    const uint32_t base = smem_u32(kind == 0 ? sm.k[0] : kind == 1 ? sm.v[0]
                                   : reinterpret_cast<uint8_t *>(lane < 8 ? sm.ks[0] : sm.vs[0]));
    const uint16_t *scales = lane < 8 ? a.p.k_scales : a.p.v_scales;
    const uint32_t row_bytes = kind < 2 ? 128 : 2, tile_row_bytes = kind < 2 ? 128 : 4;
    int issued[kStages] = {};
    Ring<kStages> r;
    bool ok = true;
    if (lane == 0 && kind < 2) prefetch_tmap(map);
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
        return lane_on && t < n && p0 < keys ? page_at(a, table, p0) : 0;
      };
      int32_t page = page_of(0);
      for (int t = 0; t < n; ++t) {
        const int32_t left = keys - (t0 + t) * kBN;
        const int valid = left < kBN ? left : kBN;
        // the page's first row in [pages, kv_heads, page_size]
        const int32_t row = (page * a.p.kv_heads + head) << a.p.page_shift;
        page = page_of(t + 1);
        if (!(ok = warp_wait(smem_u32(&sm.empty[r.slot]), r.phase ^ 1u, w))) break;
        const uint32_t bar = smem_u32(&sm.full[r.slot]);
        if (lane == 0)
          mbar_arrive_expect_tx(bar, (((valid + ps - 1) >> a.p.page_shift) << a.p.page_shift) * tile_row_bytes);
        __syncwarp();
        if (lane_on && at < valid) {
          const uint32_t dst = base + (r.slot * kBN + at) * row_bytes;
          if (kind < 2) tma_load_2d(dst, map, 0, row, bar);
          else bulk_g2s(dst, scales + row, ps * 2, bar);
        }
        ++issued[r.slot];
        r.next();
      }
    }
    // every copy that was issued must land before the CTA exits, also where a
    // consumer gives up behind the last of them
    for (int x = 0; x < kStages; ++x)
      if (issued[x]) mbar_wait_drain(smem_u32(&sm.full[x]), (issued[x] - 1) & 1, kDrainNs);
    return;
  }

  // ============================================================= consumers
  if constexpr (kBig) reg_alloc<kRegConsumer>();
  const int g8 = lane >> 2, i4 = lane & 3;   // MMA: row group and column pair
  const int key0 = warp * 16;          // its keys in a tile
  const float c2 = a.scale_log2;
  // its rows of the codes: the swizzle XORs the 16-byte chunk with row mod 8
  const uint32_t k_row = (key0 + g8) * 128, k_x = g8 & 7;
  const uint32_t v_row = (key0 + 2 * i4) * 128;
  Ring<kStages> r;
  for (;;) {
    bool ok = sr.get(sm.segs, w);
    const Seg &s = sr.seg(sm.segs);
    const int qs = sr.r.slot;
    if (ok && s.n > 0) ok = warp_wait(smem_u32(&sm.q_full[qs]), sr.r.phase, w);
    if (!kAhead && ok && s.n > 0 && warp < 2 * kNT) rotate_row(sm.q[qs][warp * 4 + (lane >> 3)], lane & 7);
    // the warps go on, or leave, together
    ok = named_bar_and(1, kWarps * 32, ok);
    if (!ok || s.n == 0) break;
    // B fragments of q'^T: of row g8 the 16 channels of chunk i4 (and i4 + 4),
    // four of them for each k step: the channel order that K's chunks give
    uint32_t qf[kBig ? 1 : kNT][16];
    auto fragments = [&](int nt, int hf, uint32_t *d) {
      const uint4 *src = reinterpret_cast<const uint4 *>(&sm.q[qs][8 * nt + g8][16 * (i4 + 4 * hf)]);
      const uint4 x = src[0], y = src[1];
      d[0] = x.x, d[1] = x.y, d[2] = x.z, d[3] = x.w, d[4] = y.x, d[5] = y.y, d[6] = y.z, d[7] = y.w;
    };
    if constexpr (!kBig) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        fragments(nt, 0, qf[nt]);
        fragments(nt, 1, qf[nt] + 8);
      }
    }
    const int32_t base_key = static_cast<int32_t>(s.keys) - s.nodes;
    float o[kNT][8][4];
    // of rows 8 nt + 2 i4 + {0, 1}: what the weights are relative to, in log2
    // units (the maximum when it was set, less kWeightLog2), and their sum
    float m[kNT][2], l[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int t = 0; t < 8; ++t) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
      m[nt][0] = m[nt][1] = kNoMaxLog2;
      l[nt][0] = l[nt][1] = 0.f;
    }
    const int32_t keys = static_cast<int32_t>(s.keys);
    const int n_tiles = s.n;
    int32_t pos = s.t0 * kBN + key0;
    for (int t = 0; t < n_tiles; ++t, pos += kBN) {
      if (!warp_wait(smem_u32(&sm.full[r.slot]), r.phase, w)) {
        ok = false;
        break;
      }
      // the step's codes and scales into registers, and the stage is free again
      uint4 kw[2][2], vw[4];
      uint32_t k0, k1, v0, v1;
      auto load_v = [&] {
        const uint8_t *vb = sm.v[r.slot] + v_row;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t row = 2 * i4 + (x & 1);  // mod 8 (keys 8 later: the same)
          vw[x] = *reinterpret_cast<const uint4 *>(vb + ((x & 1) + 8 * (x >> 1)) * 128 + ((g8 ^ row) << 4));
        }
        v0 = *reinterpret_cast<const uint32_t *>(&sm.vs[r.slot][key0 + 2 * i4]);
        v1 = *reinterpret_cast<const uint32_t *>(&sm.vs[r.slot][key0 + 2 * i4 + 8]);
        __syncwarp();
        // (a diagnostic may withhold one tile's arrival: see withhold_p_tile1)
        if (lane == 0 && t + 1 != a.withhold_p_tile1) mbar_arrive(smem_u32(&sm.empty[r.slot]));
        r.next();
      };
      {
        const uint8_t *kb = sm.k[r.slot] + k_row;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t c = ((i4 + 4 * hf) ^ k_x) << 4;
          kw[hf][0] = *reinterpret_cast<const uint4 *>(kb + c);
          kw[hf][1] = *reinterpret_cast<const uint4 *>(kb + 8 * 128 + c);
        }
        k0 = sm.ks[r.slot][key0 + g8] * 0x10001u;
        k1 = sm.ks[r.slot][key0 + g8 + 8] * 0x10001u;
      }
      if (!kBig || pos >= keys) load_v();
      if (pos < keys) {
        // S^T: keys g8 and g8 + 8, rows 2 i4 + {0, 1}; the channels in two
        // sums, so that the MMAs wait less for one another
        float st[kNT][4], su[kNT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          st[nt][0] = st[nt][1] = st[nt][2] = st[nt][3] = 0.f;
          su[nt][0] = su[nt][1] = su[nt][2] = su[nt][3] = 0.f;
        }
        if constexpr (kBig) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint4 x = kw[hf][0], y = kw[hf][1];
            uint32_t af[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t ux = (j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w) ^ 0x80808080u;
              const uint32_t uy = (j == 0 ? y.x : j == 1 ? y.y : j == 2 ? y.z : y.w) ^ 0x80808080u;
              af[j][0] = scale2(unbias(__byte_perm(ux, 0x64646464u, 0x4140)), k0);
              af[j][1] = scale2(unbias(__byte_perm(uy, 0x64646464u, 0x4140)), k1);
              af[j][2] = scale2(unbias(__byte_perm(ux, 0x64646464u, 0x4342)), k0);
              af[j][3] = scale2(unbias(__byte_perm(uy, 0x64646464u, 0x4342)), k1);
            }
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              uint32_t d[8];
              fragments(nt, hf, d);
#pragma unroll
              for (int j = 0; j < 4; ++j) mma16816(st[nt], af[j], d[2 * j], d[2 * j + 1]);
            }
          }
          load_v();
        }
#pragma unroll
        for (int j = 0; j < (kBig ? 0 : 4); ++j) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint4 x = kw[hf][0], y = kw[hf][1];
            const uint32_t ux = (j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w) ^ 0x80808080u;
            const uint32_t uy = (j == 0 ? y.x : j == 1 ? y.y : j == 2 ? y.z : y.w) ^ 0x80808080u;
            const uint32_t af[4] = {scale2(unbias(__byte_perm(ux, 0x64646464u, 0x4140)), k0),
                                    scale2(unbias(__byte_perm(uy, 0x64646464u, 0x4140)), k1),
                                    scale2(unbias(__byte_perm(ux, 0x64646464u, 0x4342)), k0),
                                    scale2(unbias(__byte_perm(uy, 0x64646464u, 0x4342)), k1)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816(hf ? su[nt] : st[nt], af, qf[kBig ? 0 : nt][8 * hf + 2 * j], qf[kBig ? 0 : nt][8 * hf + 2 * j + 1]);
          }
        }
        // scores in log2 units; keys behind the sequence and nodes off the
        // row's path do not count
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) st[nt][e] = (st[nt][e] + su[nt][e]) * c2;
        }
        if (pos + 16 > base_key) {
          const int32_t n0 = pos + g8 - base_key, n1 = n0 + 8;
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t path = sm.path[qs][8 * nt + 2 * i4 + e];
              if (n0 >= 0 && !(n0 < 64 && (path >> n0) & 1)) st[nt][e] = -INFINITY;
              if (n1 >= 0 && !(n1 < 64 && (path >> n1) & 1)) st[nt][2 + e] = -INFINITY;
            }
          }
          // scales of rows behind the sequence hold anything
          const int32_t left = keys - pos - 2 * i4;
          v0 &= left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
          v1 &= left >= 10 ? 0xffffffffu : left == 9 ? 0xffffu : 0u;
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) grow |= fmaxf(st[nt][e], st[nt][2 + e]) - m[nt][e] > kLazyRescaleLog2 + kWeightLog2;
        }
        // the maximum follows only when a score passes it by more than 2^8
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(st[nt][e], st[nt][2 + e]);
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              x = fmaxf(x - kWeightLog2, m[nt][e]);
              const float al = ex2(m[nt][e] - x);
              m[nt][e] = x;
              l[nt][e] *= al;
#pragma unroll
              for (int t8 = 0; t8 < 8; ++t8) {
                o[nt][t8][e] *= al;
                o[nt][t8][2 + e] *= al;
              }
            }
          }
        }
        uint32_t pf[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = ex2(st[nt][e] - m[nt][e & 1]);
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          pf[nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
          pf[nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
        }
        // O^T: channels 16 g8 + 2 t (+ 1) in m tile t; V'^T's pairs run along
        // the keys 2 i4 + {0, 1} (+ 8)
        const uint32_t wd[4][4] = {{vw[0].x, vw[0].y, vw[0].z, vw[0].w},
                                   {vw[1].x, vw[1].y, vw[1].z, vw[1].w},
                                   {vw[2].x, vw[2].y, vw[2].z, vw[2].w},
                                   {vw[3].x, vw[3].y, vw[3].z, vw[3].w}};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t sel = hf ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(wd[0][j], wd[1][j], sel) ^ 0x80808080u;
            const uint32_t y = __byte_perm(wd[2][j], wd[3][j], sel) ^ 0x80808080u;
            const uint32_t af[4] = {scale2(unbias(__byte_perm(x, 0x64646464u, 0x4140)), v0),
                                    scale2(unbias(__byte_perm(x, 0x64646464u, 0x4342)), v0),
                                    scale2(unbias(__byte_perm(y, 0x64646464u, 0x4140)), v1),
                                    scale2(unbias(__byte_perm(y, 0x64646464u, 0x4342)), v1)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mma16816(o[nt][2 * j + hf], af, pf[nt][0], pf[nt][1]);
          }
        }
      }
    }
    // join the warps: common maximum, then the sum of the rescaled parts in order
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g8 == 0) {
          sm.m[warp][8 * nt + 2 * i4 + e] = m[nt][e];
          sm.l[warp][8 * nt + 2 * i4 + e] = x;
        }
      }
    }
    if (!named_bar_and(1, kWarps * 32, ok)) break;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nt + 2 * i4 + e;
        float top = sm.m[0][row];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) top = fmaxf(top, sm.m[x][row]);
        const float f = ex2(m[nt][e] - top);
        float4 *dst = reinterpret_cast<float4 *>(&sm.o[warp][2 * i4 + e][16 * g8]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dst[j] = make_float4(o[nt][2 * j][e] * f, o[nt][2 * j][2 + e] * f, o[nt][2 * j + 1][e] * f,
                               o[nt][2 * j + 1][2 + e] * f);
      }
      named_bar_sync(1, kWarps * 32);
      const int row = 8 * nt + warp;
      if (row < s.rows) {
        float top = sm.m[0][row], sum = 0.f;
#pragma unroll
        for (int x = 1; x < kWarps; ++x) top = fmaxf(top, sm.m[x][row]);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) sum = fmaf(sm.l[x][row], ex2(sm.m[x][row] - top), sum);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float4 y = *reinterpret_cast<const float4 *>(&sm.o[x][warp][4 * lane]);
          v[0] += y.x;
          v[1] += y.y;
          v[2] += y.z;
          v[3] += y.w;
        }
        if (s.whole) {
          const int x = s.row0 + row, node = node_of(a, x), h = s.head * a.group + (x - node * a.group);
          fwht128_warp(v, lane);
          const float inv = kInvSqrt128 / sum;
          *reinterpret_cast<uint2 *>(a.o.data + h * a.o.head_stride + (s.q_base + node) * a.o.row_stride + 4 * lane) =
              make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
          if (a.lse && lane == 0) a.lse[h * a.nodes + s.q_base + node] = kLn2 * (top + log2f(sum));
        } else {
          const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + (s.t0 > 0 ? 0 : 1)) * ws.rows + row;
          reinterpret_cast<float4 *>(ws.o + at * 128)[lane] = make_float4(v[0], v[1], v[2], v[3]);
          if (lane == 0) ws.ml[at] = make_float2(top / c2, sum);
        }
      }
      named_bar_sync(1, kWarps * 32);
    }
    sr.done(sm.segs);
  }
}

template <int kNT>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const TreeArgs &a, cudaStream_t stream) {
  constexpr int kBytes = sizeof(FewSmem<kNT>) + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_smem(few_kernel<kNT>, kBytes, allowed);
  if (e != cudaSuccess) return e;
  few_kernel<kNT><<<a.ctas, kFewThreads, kBytes, stream>>>(tk, tv, a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace serve

cudaError_t launch_tree_few(const TreeArgs &a, cudaStream_t stream) {
  const int64_t rows = (static_cast<int64_t>(a.p.pages) * a.p.kv_heads) << a.p.page_shift;
  CUtensorMap tk, tv;
  if (!encode_codes(&tk, a.p.k_codes, rows, a.p.page_size) || !encode_codes(&tv, a.p.v_codes, rows, a.p.page_size))
    return cudaErrorInvalidValue;
  return a.item_rows == 8    ? serve::launch<1>(tk, tv, a, stream)
         : a.item_rows == 16 ? serve::launch<2>(tk, tv, a, stream)
                             : serve::launch<4>(tk, tv, a, stream);
}

}  // namespace h3kv
