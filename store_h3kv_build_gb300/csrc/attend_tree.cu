// attend_tree.cu -- attention of drafted tokens over the paged kvi8r cache: the
// kernel for many rows of a sequence and kv head (the tcgen05 pipeline of
// serve_attend.cuh), the join, and the choice of kernel.
#include "tree.cuh"

namespace h3kv {
namespace serve {
namespace {

struct TreeSmem : Smem {
  Scan scan;
};
constexpr size_t kTreeSmemBytes = sizeof(TreeSmem) + 1024;
static_assert(kTreeSmemBytes <= 232448, "shared memory budget");

__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  TreeSmem &sm = *reinterpret_cast<TreeSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Workspace ws = workspace_of(a);

  // the join may start its CTAs; it waits there until this grid is done
  if (tid == 0) pdl_launch_dependents();
  find_run<kThreads>(a, ws, sm.scan);
  if (sm.scan.u0 >= sm.scan.u1) return;

  if (tid == 0) init_barriers(sm, true);
  if (warp == 13) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const WaitCtx w{a.p.err, &sm.abort, a.timeout_ns};
  Walk walk;
  Seg s;

  if (warp < 8) {
    // =================================================== softmax warpgroups
    reg_alloc<kRegSoftmax>();
    walk.start(a, sm.scan);
    const int q = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + q * 128, tO = tmem + lane_base + 256 + q * 128;
    const float c2 = a.scale_log2;
    const int i = tid & 127;
    uint32_t s_phase = 0, o_phase = 0;
    while (walk.next(a, &s)) {
      const int base_row = s.two ? q * kBM : 0;
      const int r = base_row + i;
      const int w0 = base_row + (warp & 3) * 32;  // the warp's first row
      const bool warp_on = w0 < s.rows;
      // q' = fp16(q H) into the swizzled K-major tile, which is free: this
      // stream's last QK of the segment before has completed.  8 lanes hold a
      // row (values 8l .. 8l+7 and 64 + 8l .. of it), the warp 4 rows at a
      // time; all of its rows' loads go out before the first is used.
      if (has_tiles(s, q)) {
        if (warp_on) {
          const int l = lane & 7;
          uint4 raw[8][2];
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int rr = it * 4 + (lane >> 3);
            raw[it][0] = raw[it][1] = make_uint4(0, 0, 0, 0);
            if (w0 + rr < s.rows) {
              const int x = s.row0 + w0 + rr, node = x / a.group, h = s.head * a.group + (x - node * a.group);
              const uint4 *src = reinterpret_cast<const uint4 *>(a.q.data + h * a.q.head_stride +
                                                                 (s.q_base + node) * a.q.row_stride) +
                                 l;
              raw[it][0] = __ldg(src);
              raw[it][1] = __ldg(src + 8);
            }
          }
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            if (w0 + it * 4 >= s.rows) break;
            const int rr = (warp & 3) * 32 + it * 4 + (lane >> 3);
            float v[16];
            unpack_bf16x8(raw[it][0], v);
            unpack_bf16x8(raw[it][1], v + 8);
            fwht128_oct(v, l);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= kInvSqrt128;
#pragma unroll
            for (int hi = 0; hi < 2; ++hi)
              *reinterpret_cast<uint4 *>(sm.q[q] + hi * kChunkBytes + sw128_off(rr, l)) =
                  make_uint4(pack_f16x2(v[8 * hi], v[8 * hi + 1]), pack_f16x2(v[8 * hi + 2], v[8 * hi + 3]),
                             pack_f16x2(v[8 * hi + 4], v[8 * hi + 5]), pack_f16x2(v[8 * hi + 6], v[8 * hi + 7]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[q]));
      }
      const int32_t len = static_cast<int32_t>(s.keys), base_key = len - s.nodes;
      uint64_t path = 0;
      if (r < s.rows) path = path_of(a, s.q_base, (s.row0 + r) / a.group);
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
          const int32_t pos = (s.t0 + t) * kBN;
          const bool masked = pos + kBN > base_key;
          uint32_t see[4];
          tree_mask(pos, base_key, path, see);
          softmax_tile<true>(tS, tO, t == t_first, masked, see, c2, row);
        }
        tc_fence_before();
        __syncwarp();
        // (a diagnostic may withhold one tile's arrival: see withhold_p_tile1)
        if (lane == 0 && t + 1 != a.withhold_p_tile1) mbar_arrive(smem_u32(&sm.p_full[q]));
      }
      ok = ok && warp_wait(smem_u32(&sm.o_full), o_phase, w);
      o_phase ^= 1u;
      tc_fence_after();
      if (!s.two && q == 1) sm.ml[i] = make_float2(row.m, row.l);
      ok = named_bar_and(1, 256, ok);
      if (!ok) break;
      if ((s.two || q == 0) && warp_on) {
        const bool joined = !s.two && s.n > 1;
        float ga = 1.f, gb = 0.f;
        if (joined) join_rows(row, sm.ml[i], c2, ga, gb);
        float o[128];
        if (s.whole) {
          const float inv = kInvSqrt128 / row.l;
          load_o(tO, tO + 128, joined, ga * inv, gb * inv, o);
          fwht128_packed(o);
          if (r < s.rows) {
            const int x = s.row0 + r, node = x / a.group, h = s.head * a.group + (x - node * a.group);
            uint4 *dst = reinterpret_cast<uint4 *>(a.o.data + h * a.o.head_stride +
                                                   (s.q_base + node) * a.o.row_stride);
#pragma unroll
            for (int g = 0; g < 16; ++g)
              dst[g] = make_uint4(pack_bf16x2(o[8 * g], o[8 * g + 1]), pack_bf16x2(o[8 * g + 2], o[8 * g + 3]),
                                  pack_bf16x2(o[8 * g + 4], o[8 * g + 5]), pack_bf16x2(o[8 * g + 6], o[8 * g + 7]));
            if (a.lse) a.lse[h * a.nodes + s.q_base + node] = kLn2 * (row.m * c2 + log2f(row.l));
          }
        } else {
          load_o(tO, tO + 128, joined, ga, gb, o);
          if (r < s.rows) {
            const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + (s.t0 > 0 ? 0 : 1)) * ws.rows + r;
            float4 *dst = reinterpret_cast<float4 *>(ws.o + at * 128);
#pragma unroll
            for (int g = 0; g < 32; ++g) dst[g] = make_float4(o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]);
            ws.ml[at] = make_float2(row.m, row.l);
          }
        }
      }
      // stream 1's O and (max, sum) have been read
      if (!s.two) named_bar_sync(2, 256);
      tc_fence_before();
    }
  } else if (warp < 12) {
    // ======================================================= dequantisers
    reg_dealloc<kRegDequant>();
    walk.start(a, sm.scan);
    const int dw = warp - 8;
    const attn::DqOffsets off = attn::dq_offsets(dw, lane);
    const int rr = 2 * (lane >> 4) + ((lane >> 2) & 1);
    Ring<kNK> kr;
    Ring<kNV> vr;
    // The tile's 128 scales lie in the buffer's first half, each warp's 32 in
    // the 64 bytes at its own first row: read by the whole warp before any of
    // its lanes writes there.  Rows behind the sequence get scale 0.
    auto dequant = [&](uint8_t *tile, int valid) {
      const uint16_t *p = reinterpret_cast<const uint16_t *>(tile + dw * 32 * 128) + rr;
      uint16_t sc[8];
#pragma unroll
      for (int it = 0; it < 8; ++it) sc[it] = dw * 32 + rr + 4 * it < valid ? p[4 * it] : 0;
      __syncwarp();
      attn::dequant_tile(tile, sc, off);
      fence_proxy_async_smem();
      __syncwarp();
    };
    bool ok = true;
    while (ok && walk.next(a, &s)) {
      for (int t = 0; t < s.n; ++t) {
        const int64_t left = s.keys - static_cast<int64_t>(s.t0 + t) * kBN;
        const int valid = left < kBN ? static_cast<int>(left) : kBN;
        if (!(ok = warp_wait(smem_u32(&sm.k_load[kr.slot]), kr.phase, w))) break;
        dequant(sm.k[kr.slot], valid);
        if (lane == 0) mbar_arrive(smem_u32(&sm.k_ready[kr.slot]));
        kr.next();
        if (!(ok = warp_wait(smem_u32(&sm.v_load[vr.slot]), vr.phase, w))) break;
        dequant(sm.v[vr.slot], valid);
        if (lane == 0) mbar_arrive(smem_u32(&sm.v_ready[vr.slot]));
        vr.next();
      }
    }
  } else {
    reg_dealloc<kRegIssue>();
    walk.start(a, sm.scan);
    if (warp == 12) {
      // ========================================================== producer
      // A tile's codes come page by page (lanes 0-7) into the buffer's second
      // half, its scales in pieces of at most 32 (lanes 8-15) into the first.
      const int ps = a.p.page_size, sp = ps < 32 ? ps : 32;
      const bool codes = lane < 8;
      const int piece = lane & 7;
      const int at = piece * (codes ? ps : sp);  // the piece's first row in the tile
      int k_issued[kNK] = {0, 0, 0}, v_issued[kNV] = {0, 0};
      Ring<kNK> kr;
      Ring<kNV> vr;
      bool ok = true;
      while (ok && walk.next(a, &s)) {
        for (int t = 0; t < s.n; ++t) {
          const int32_t pos = (s.t0 + t) * kBN;
          const int64_t left = s.keys - pos;
          const int valid = left < kBN ? static_cast<int>(left) : kBN;
          const bool on = lane < 16 && at < valid;
          int64_t src = 0;
          uint32_t bytes = 0, dst = 0;
          if (on) {
            const int32_t page = page_at(a, s.k_base, pos + at);
            src = ((static_cast<int64_t>(page) * a.p.kv_heads + s.head) << a.p.page_shift) +
                  ((pos + at) & (ps - 1));
            if (codes) {
              const int n = valid - at < ps ? valid - at : ps;
              bytes = n * 128;
              dst = kChunkBytes + at * 128;
            } else {
              bytes = sp * 2;
              dst = (at >> 5) * 32 * 128 + (at & 31) * 2;
            }
          }
          uint32_t sum = bytes;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          if (!(ok = warp_wait(smem_u32(&sm.k_free[kr.slot]), kr.phase ^ 1u, w))) break;
          uint32_t bar = smem_u32(&sm.k_load[kr.slot]);
          if (lane == 0) mbar_arrive_expect_tx(bar, sum);
          __syncwarp();
          if (on)
            bulk_g2s(smem_u32(sm.k[kr.slot]) + dst,
                     codes ? static_cast<const void *>(a.p.k_codes + src * 128)
                           : static_cast<const void *>(a.p.k_scales + src),
                     bytes, bar);
          ++k_issued[kr.slot];
          kr.next();
          if (!(ok = warp_wait(smem_u32(&sm.v_free[vr.slot]), vr.phase ^ 1u, w))) break;
          bar = smem_u32(&sm.v_load[vr.slot]);
          if (lane == 0) mbar_arrive_expect_tx(bar, sum);
          __syncwarp();
          if (on)
            bulk_g2s(smem_u32(sm.v[vr.slot]) + dst,
                     codes ? static_cast<const void *>(a.p.v_codes + src * 128)
                           : static_cast<const void *>(a.p.v_scales + src),
                     bytes, bar);
          ++v_issued[vr.slot];
          vr.next();
        }
      }
      if (sm.abort) {
        // every copy that was issued must land before the CTA exits
        for (int x = 0; x < kNK; ++x)
          if (k_issued[x]) mbar_wait_drain(smem_u32(&sm.k_load[x]), (k_issued[x] - 1) & 1, kDrainNs);
        for (int x = 0; x < kNV; ++x)
          if (v_issued[x]) mbar_wait_drain(smem_u32(&sm.v_load[x]), (v_issued[x] - 1) & 1, kDrainNs);
      }
    } else if (warp == 13) {
      MmaState m;
      mma_setup(m, sm, false);
      while (walk.next(a, &s))
        if (!mma_segment<true>(m, sm, s, false, w)) break;
      // every MMA issued must finish before TMEM is released
      mma_commit(m.go, smem_u32(&sm.drain));
      mbar_wait_drain(smem_u32(&sm.drain), 0, kDrainNs);
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

// One warp for an output row (a node of a query head): joins the parts of its
// item over the CTAs that worked on it, in order, un-rotates and writes.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const TreeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  const int64_t row = unit / a.q_heads;
  const int h = static_cast<int>(unit - row * a.q_heads);
  int lo = 0, hi = row < a.nodes ? a.seqs : 0;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_nodes + mid + 1) <= row) lo = mid + 1;
    else hi = mid;
  }
  const bool live = row < a.nodes && lo < a.seqs;
  Counts c = {};
  if (live) c = counts_of(a, lo);
  // (no thread leaves before this, so the grids end in stream order)
  pdl_wait_prerequisites();
  if (!live || c.units == 0 || row < c.q_base || row >= c.q_base + c.nodes) return;
  const Workspace ws = workspace_of(a);
  const int64_t total = ws.prefix[a.seqs];
  const int head = h / a.group;
  const int x = static_cast<int>(row - c.q_base) * a.group + (h - head * a.group);
  const int rt = x / a.item_rows, r = x - rt * a.item_rows;
  const int64_t u0 = ws.prefix[lo] + (static_cast<int64_t>(head) * c.row_tiles + rt) * c.tiles, u1 = u0 + c.tiles;
  // the CTA that holds unit u: the last with first_unit <= u
  const int ctas = working(a, total);
  auto owner = [&](int64_t u) {
    int k = static_cast<int>(u * ctas / total);
    while (k + 1 < ctas && first_unit(total, k + 1, ctas) <= u) ++k;
    while (k > 0 && first_unit(total, k, ctas) > u) --k;
    return k;
  };
  const int first = owner(u0), last = owner(u1 - 1);
  if (first == last) return;  // written by the attention kernel
  float m = kNoMax, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = first; k <= last; ++k) {
    const int64_t at = (static_cast<int64_t>(k) * 2 + (k == first ? 1 : 0)) * ws.rows + r;
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
  const int64_t units = a.nodes * a.q_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((units + kJoinWarps - 1) / kJoinWarps));
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
