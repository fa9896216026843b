// attend_tree.cu -- attention of drafted tokens over the paged kvi8r cache: the
// kernel for many rows of a sequence and kv head (the tcgen05 pipeline of
// serve_attend.cuh), the join, and the choice of kernel.
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
  if (sm.abort) {
    // every copy that was issued must land before the CTA exits
    for (int x = 0; x < kDepth; ++x)
      if (issued[x]) mbar_wait_drain(smem_u32(&load[x]), (issued[x] - 1) & 1, kDrainNs);
  }
}

__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  TreeSmem &sm = *reinterpret_cast<TreeSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Workspace ws = workspace_of(a);

  // the join may start its CTAs; it waits there until this grid is done
  if (tid == 0) pdl_launch_dependents();
  find_run<kThreads>(a, ws, sm.scan);
  if (sm.scan.u0 >= sm.scan.u1) return;

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
    uint32_t s_phase = 0, o_phase = 0;
    for (;;) {
      // the eight warps go on, or leave, together
      if (!named_bar_and(1, 256, sr.get(sm.segs, w))) break;
      const Seg &s = sr.seg(sm.segs);
      if (s.n == 0) break;
      const int base_row = s.two ? q * kBM : 0;
      const int r = base_row + i;
      const int w0 = base_row + (warp & 3) * 32;  // the warp's first row
      const bool warp_on = w0 < s.rows;
      // q' = fp16(q H) into the swizzled K-major tile, which is free: this
      // stream's last QK of the segment before has completed.  A thread takes
      // its own row: H128 = [[H64, H64], [H64, -H64]], so half hf of the
      // rotated row is H64 of the sum (hf 0) or difference (hf 1) of the row's
      // halves, 64 values in registers and no shuffles (with a row over 8
      // lanes they took most of 5 us); a loop over hf, since instructions that
      // run once a segment are waited for.
      if (has_tiles(s, q)) {
        if (warp_on) {
          uint4 raw[16];
          const int x = s.row0 + r, node = node_of(a, x), h = s.head * a.group + (x - node * a.group);
          const uint4 *src =
              reinterpret_cast<const uint4 *>(a.q.data + h * a.q.head_stride + (s.q_base + node) * a.q.row_stride);
#pragma unroll
          for (int g = 0; g < 16; ++g) raw[g] = r < s.rows ? __ldg(src + g) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            const float2 sign = hf ? make_float2(-1.f, -1.f) : make_float2(1.f, 1.f);
            float v[64];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              float lo[8], hi[8];
              unpack_bf16x8(raw[g], lo);
              unpack_bf16x8(raw[8 + g], hi);
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 y = __ffma2_rn(make_float2(hi[e], hi[e + 1]), sign, make_float2(lo[e], lo[e + 1]));
                v[8 * g + e] = y.x;
                v[8 * g + e + 1] = y.y;
              }
            }
            fwht64_packed(v);
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] *= kInvSqrt128;
#pragma unroll
            for (int g = 0; g < 8; ++g)
              *reinterpret_cast<uint4 *>(sm.q[q] + hf * kChunkBytes + sw128_off(i, g)) =
                  make_uint4(pack_f16x2(v[8 * g], v[8 * g + 1]), pack_f16x2(v[8 * g + 2], v[8 * g + 3]),
                             pack_f16x2(v[8 * g + 4], v[8 * g + 5]), pack_f16x2(v[8 * g + 6], v[8 * g + 7]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
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
            softmax_tile<true, true>(tS, tO, t == t_first, see, c2, row);
          } else {
            softmax_tile<true, false>(tS, tO, t == t_first, see, c2, row);
          }
        }
        tc_fence_before();
        __syncwarp();
        // (a diagnostic may withhold one tile's arrival: see withhold_p_tile1)
        if (lane == 0 && t + 1 != a.withhold_p_tile1) mbar_arrive(smem_u32(&sm.p_full[q]));
      }
      ok = ok && warp_wait(smem_u32(&sm.o_full), o_phase, w);
      o_phase ^= 1u;
      tc_fence_after();
      if (!s.two && q == 1) join_ml(sm)[i] = make_float2(row.m, row.l);
      ok = named_bar_and(1, 256, ok);
      if (!ok) break;
      if ((s.two || q == 0) && warp_on) {
        const bool joined = !s.two && s.n > 1;
        float ga = 1.f, gb = 0.f;
        if (joined) join_rows(row, join_ml(sm)[i], c2, ga, gb);
        // the rows go out through this stream's Q tile (free until the next
        // segment's rows are written), 16-byte granule g of a row at
        // g ^ (row mod 16), so that a warp writes whole rows
        float o[128];
        uint8_t *stage = sm.q[q] + i * 256;
        const int g = lane & 15;
        const float inv = s.whole ? kInvSqrt128 / row.l : 1.f;
        load_o(tO, tO + 128, joined, ga * inv, gb * inv, o);
        if (s.whole) {
          fwht128_packed(o);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            *reinterpret_cast<uint4 *>(stage + ((k ^ (i & 15)) << 4)) =
                make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                           pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
          __syncwarp();
          for (int rr = 0; rr < 32; rr += 2) {
            const int ti = rr + (lane >> 4);
            if (w0 + ti < s.rows) {
              const int x = s.row0 + w0 + ti, node = node_of(a, x), h = s.head * a.group + (x - node * a.group);
              const int sr_row = (warp & 3) * 32 + ti;
              *reinterpret_cast<uint4 *>(a.o.data + h * a.o.head_stride + (s.q_base + node) * a.o.row_stride + g * 8) =
                  *reinterpret_cast<const uint4 *>(sm.q[q] + sr_row * 256 + ((g ^ (sr_row & 15)) << 4));
            }
          }
          if (a.lse && r < s.rows) {
            const int x = s.row0 + r, node = node_of(a, x), h = s.head * a.group + (x - node * a.group);
            a.lse[h * a.nodes + s.q_base + node] = kLn2 * (row.m * c2 + log2f(row.l));
          }
        } else {
          const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + (s.t0 > 0 ? 0 : 1)) * ws.rows;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              *reinterpret_cast<float4 *>(stage + ((k ^ (i & 15)) << 4)) =
                  make_float4(o[64 * hf + 4 * k], o[64 * hf + 4 * k + 1], o[64 * hf + 4 * k + 2], o[64 * hf + 4 * k + 3]);
            __syncwarp();
            for (int rr = 0; rr < 32; rr += 2) {
              const int ti = rr + (lane >> 4), sr_row = (warp & 3) * 32 + ti;
              if (w0 + ti < s.rows)
                *reinterpret_cast<float4 *>(ws.o + (at + w0 + ti) * 128 + 64 * hf + 4 * g) =
                    *reinterpret_cast<const float4 *>(sm.q[q] + sr_row * 256 + ((g ^ (sr_row & 15)) << 4));
            }
            __syncwarp();
          }
          if (r < s.rows) ws.ml[at + r] = make_float2(row.m, row.l);
        }
      }
      // stream 1's O and (max, sum) have been read
      if (!s.two) named_bar_sync(2, 256);
      tc_fence_before();
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
    bool ok = true;
    while (ok && (ok = sr.get(sm.segs, w))) {
      const Seg &s = sr.seg(sm.segs);
      const int n = s.n, head = s.head;
      const int64_t table = s.k_base;
      const int32_t keys = static_cast<int32_t>(s.keys);
      int32_t pos = s.t0 * kBN + dw * 32;  // the warp's first row
      sr.done(sm.segs);
      if (n == 0) break;
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
      publish_segments(a, sm.scan, sm.segs, w);
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

// Joins the items that lie on several CTAs: CTA column b takes the item that the
// b-th CTA goes on with, where that CTA is the item's second.  One warp for a
// row: its parts in order, un-rotated and written.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const TreeArgs a) {
  const int lane = threadIdx.x & 31, b = blockIdx.x + 1;
  // (no thread leaves before this, so the grids end in stream order)
  pdl_wait_prerequisites();
  const Workspace ws = workspace_of(a);
  const int64_t total = ws.prefix[a.seqs];
  const int ctas = working(a, total);
  if (b >= ctas) return;
  const int64_t u = first_unit(total, b, ctas);
  // the sequence that holds unit u: the last with prefix <= u (those without
  // work share theirs with the next)
  int lo = 0, hi = a.seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ws.prefix[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  const Counts c = counts_of(a, lo);
  const int size = c.tiles + a.item_cost;
  const int64_t item = (u - ws.prefix[lo]) / size;
  // its tiles' units, and the first CTA that has one
  const int64_t u0 = ws.prefix[lo] + item * size + a.item_cost, u1 = u0 + c.tiles;
  if (u <= u0 || first_unit(total, b - 1, ctas) > u0) return;
  const int head = static_cast<int>(item / c.row_tiles);
  const int row0 = static_cast<int>(item - static_cast<int64_t>(head) * c.row_tiles) * a.item_rows;
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int x = row0 + r;
  if (r >= a.item_rows || x >= c.nodes * a.group) return;
  float m = kNoMax, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = b - 1; k < ctas && first_unit(total, k, ctas) < u1; ++k) {
    const int64_t at = (static_cast<int64_t>(k) * 2 + (k == b - 1 ? 1 : 0)) * ws.rows + r;
    const float2 ml = ws.ml[at];
    const float4 p = reinterpret_cast<const float4 *>(ws.o + at * 128)[lane];
    const float mn = fmaxf(m, ml.x);
    const float ga = ex2((m - mn) * a.scale_log2), gb = ex2((ml.x - mn) * a.scale_log2);
    l = fmaf(l, ga, ml.y * gb);
    o[0] = fmaf(o[0], ga, p.x * gb);
    o[1] = fmaf(o[1], ga, p.y * gb);
    o[2] = fmaf(o[2], ga, p.z * gb);
    o[3] = fmaf(o[3], ga, p.w * gb);
    m = mn;
  }
  fwht128_warp(o, lane);
  const float inv = kInvSqrt128 / l;
  const int node = node_of(a, x), h = head * a.group + (x - node * a.group);
  const int64_t row = c.q_base + node;
  *reinterpret_cast<uint2 *>(a.o.data + h * a.o.head_stride + row * a.o.row_stride + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse && lane == 0) a.lse[h * a.nodes + row] = kLn2 * (m * a.scale_log2 + log2f(l));
}

}  // namespace
}  // namespace serve

size_t tree_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t nodes, int32_t seqs) {
  const int32_t group = q_heads / kv_heads;
  const size_t rows = serve::part_rows(group, nodes, serve::item_rows_of(group, nodes, seqs));
  return serve::prefix_bytes(seqs) + serve::kMaxCtas * 2 * rows * (128 * sizeof(float) + sizeof(float2));
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
    e = cudaFuncSetAttribute(tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kTreeSmemBytes));
    if (e != cudaSuccess) return e;
    tree_kernel<<<a.ctas, kThreads, kTreeSmemBytes, stream>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  if (a.ctas < 2) return cudaSuccess;
  const int rows = part_rows(a.group, a.nodes, a.item_rows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas - 1, (rows + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, a);
}

}  // namespace h3kv
