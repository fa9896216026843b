// attend_tree.cu -- attention of drafted tokens over the paged kvi8r cache: the
// kernel for many rows of a sequence and kv head (the tcgen05 pipeline of
// serve_attend.cuh), the join, and the choice of kernel.
//
// Bound by shared memory, which feeds the products and carries the codes and
// their fp16 values, and by the issue slots that dequantisation and softmax
// share: 1.9 us for 256 rows over a 128-key tile, where the products alone take
// 1.3 (the tensor rate) and the bytes 0.75.  A segment costs some 12 us more
// before its first tile (counts, query rows, first page) and 4 behind its last.
// A thread spills 56 bytes.  Measured at 64 nodes, 32 query heads over 8: 2 x
// 131072 cached rows 228 us (1207 TFLOP/s), 32 x 8192 250 us, 128 x 2048 334 us,
// 512 x 512 506 us.
#include "store_fwht.cuh"
#include "tree.cuh"

namespace h3kv {
namespace serve {
namespace {

struct TreeSmem : Smem {
  Scan scan;
  TreeSegs segs;
};
constexpr size_t kTreeSmemBytes = sizeof(TreeSmem) + 1024;
static_assert(kTreeSmemBytes <= 232448, "shared memory budget");

// The producer warp of K or of V: a tile's codes, one copy per page (lanes 0-7),
// into the second half of the tile's buffer.  (Copies are what a producer has
// too little time for: with the scales copied too, in pieces of 32, the kernel
// took half as long again.)
template <int kDepth>
__device__ __forceinline__ void produce(const TreeArgs &a, TreeSmem &sm, uint8_t (&ring)[kDepth][kTileBytes],
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

// q' = fp16(q H) of 32 rows of a segment, from row w0 on, into rows t0 .. of the
// swizzled K-major tile; zeros behind the segment's rows.  One warp: 8 lanes
// hold a row (values 8l .. 8l+7 and 64 + 8l .. of it), 4 rows at a time.  The
// rows are copied as they are to the places where the same lanes then write
// them rotated.  Loops that are not unrolled: instructions that run once a
// segment are waited for (unrolled, this took 10 us).
__device__ __forceinline__ void rotate_rows(const TreeArgs &a, const Seg &s, uint8_t *tile, int w0, int t0) {
  const int lane = threadIdx.x & 31, l = lane & 7, ti = t0 + (lane >> 3);
  if (w0 < s.rows) {
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
      const int row = w0 + it * 4 + (lane >> 3);
      const bool in = row < s.rows;
      const int x = s.row0 + (in ? row : 0), node = node_of(a, x), h = s.head * a.group + (x - node * a.group);
      const uint16_t *src = a.q.data + h * a.q.head_stride + (s.q_base + node) * a.q.row_stride + 8 * l;
      const uint32_t dst = smem_u32(tile) + sw128_off(ti + 4 * it, l);
      copy16_async(dst, src, in);
      copy16_async(dst + kChunkBytes, src + 64, in);
    }
    copy16_wait();
#pragma unroll 1
    for (int it = 0; it < 8 && w0 + it * 4 < s.rows; ++it) {
      uint4 *lo = reinterpret_cast<uint4 *>(tile + sw128_off(ti + 4 * it, l));
      uint4 *hi = reinterpret_cast<uint4 *>(tile + kChunkBytes + sw128_off(ti + 4 * it, l));
      float v[16];
      unpack_bf16x8(*lo, v);
      unpack_bf16x8(*hi, v + 8);
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

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  TreeSmem &sm = *reinterpret_cast<TreeSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Workspace ws = workspace_of(a);

  // the join may start its CTAs; it waits there until this grid is done
  if (tid == 0) pdl_launch_dependents();
  find_run<kThreads>(a, sm.scan, reinterpret_cast<int64_t *>(sm.q[0]));
  if (sm.scan.u0 >= sm.scan.u1) {
    if (tid == 0) ws.split[blockIdx.x].parts = 0;
    return;
  }

  if (tid == 0) {
    init_seg_ring(sm.segs, 15);
    init_barriers(sm, true);
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
    const float c2 = a.scale_log2;
    const int i = tid & 127;
    uint32_t s_phase = 0;
    bool first = true;
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
          rotate_rows(a, s, sm.q[q], w0, (warp & 3) * 32);
          if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
        }
      }
      const int32_t base_key = static_cast<int32_t>(s.keys) - s.nodes, pos0 = s.t0 * kBN;
      uint64_t path = 0;
      if (r < s.rows) path = path_of(a, s.q_base, node_of(a, s.row0 + r));
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
          if (pos + kBN > base_key) {
            tree_mask(pos, base_key, path, see);
            mask_tile(tS, see);
          }
          softmax_tile<true>(tS, tO, t == t_first, c2, row);
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
        if (s.whole) {
          // H128 = [[H64, H64], [H64, -H64]]: the output's halves are the
          // transforms of the sum and of the difference of O's; a loop over
          // them (code of half the size, see mask_tile)
          const float inv = kInvSqrt128 / row.l, gx = ga * inv, gy = gb * inv;
          const int x = s.row0 + r, node = node_of(a, live ? x : 0), h = s.head * a.group + (x - node * a.group);
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
      sr.done(sm.segs);
    }
  } else if (warp < 12) {
    // ======================================================= dequantisers
    reg_dealloc<kRegDequant>();
    const int dw = warp - 8;
    const attn::DqOffsets off = attn::dq_offsets(dw, lane);
    const int rr = 2 * (lane >> 4) + ((lane >> 2) & 1);
    Ring<kNK> kr;
    Ring<kNV> vr;
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
        rotate_rows(a, s, sm.q[q], (s.two ? q * kBM : 0) + dw * 32, dw * 32);
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
      }
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
      produce<kNK>(a, sm, sm.k, sm.k_load, sm.k_free, a.p.k_codes, w);
    } else if (warp == 14) {
      produce<kNV>(a, sm, sm.v, sm.v_load, sm.v_free, a.p.v_codes, w);
    } else if (warp == 13) {
      MmaState m;
      mma_setup(m, sm, false);
      while (sr.get(sm.segs, w)) {
        const Seg s = sr.seg(sm.segs);
        sr.done(sm.segs);
        if (s.n == 0 || !mma_segment<true>(m, sm, s, false, w)) break;
      }
      // every MMA issued must finish before TMEM is released
      mma_commit(m.go, smem_u32(&sm.drain));
      mbar_wait_drain(smem_u32(&sm.drain), 0, kDrainNs);
    } else if (warp == 15) {
      publish_segments(a, sm.scan, ws, sm.segs, w, [](const Seg &, int) { return true; });
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
__global__ void __launch_bounds__(kJoinWarpsFew * 32) join_kernel(const TreeArgs a) {
  extern __shared__ float4 sh_o[];  // [warps][4][32], if the warps share parts
  __shared__ float2 sh_ml[kJoinWarpsFew][kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x + 1;
  const int l8 = lane & 7, sub = lane >> 3, warps = blockDim.x >> 5;
  // (no thread leaves before this, so the grids end in stream order)
  pdl_wait_prerequisites();
  const Workspace ws = workspace_of(a);
  const Split sp = ws.split[b];
  if (sp.parts == 0) return;
  const int lg = ws.rows <= 4 ? 0 : ws.rows <= 8 ? 1 : ws.rows <= 16 || warps == 4 ? 2 : 3, groups = 1 << lg, ways = warps >> lg;
  const int g = warp & (groups - 1), way = warp >> lg;
  const int r = (blockIdx.y * groups + g) * kJoinRows + sub;
  const bool live = r < sp.rows;
  const float c2 = a.scale_log2;
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
  fwht128_oct(o, l8);
  if (!live) return;
  const float inv = kInvSqrt128 / l;
  const int x = sp.row0 + r, node = node_of(a, x), h = sp.head * a.group + (x - node * a.group);
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

}  // namespace
}  // namespace serve

size_t tree_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t nodes, int32_t seqs) {
  const int32_t group = q_heads / kv_heads;
  const size_t rows = serve::part_rows(group, nodes, serve::item_rows_of(group, nodes, seqs));
  return serve::kMaxCtas * (sizeof(serve::Split) + 2 * rows * (128 * sizeof(float) + sizeof(float2)));
}

cudaError_t launch_attend_tree(const TreeArgs &args, cudaStream_t stream) {
  using namespace serve;
  TreeArgs a = args;
  a.ctas = a.ctas < kMaxCtas ? a.ctas : kMaxCtas;
  a.item_rows = item_rows_of(a.group, a.nodes, a.seqs);
  a.item_cost = item_cost_of(a.item_rows);
  a.group_magic = ((1u << 19) + a.group - 1) / a.group;
  cudaError_t e;
  if (a.item_rows < kManyRows) {
    e = launch_tree_few(a, stream);
  } else {
    // whole 32-byte sectors per store where the output's alignment allows
    const bool wide = ((reinterpret_cast<uintptr_t>(a.o.data) | static_cast<uintptr_t>(a.o.head_stride * 2) |
                        static_cast<uintptr_t>(a.o.row_stride * 2)) &
                       31) == 0;
    auto kernel = wide ? tree_kernel<true> : tree_kernel<false>;
    static std::atomic<uint64_t> allowed[2];
    e = allow_smem(kernel, static_cast<int>(kTreeSmemBytes), allowed[wide]);
    if (e != cudaSuccess) return e;
    kernel<<<a.ctas, kThreads, kTreeSmemBytes, stream>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  if (a.ctas < 2) return cudaSuccess;
  const int rows = part_rows(a.group, a.nodes, a.item_rows);
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
  return cudaLaunchKernelEx(&cfg, join_kernel, a);
}

}  // namespace h3kv
