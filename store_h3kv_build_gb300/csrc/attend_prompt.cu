// attend_prompt.cu -- attention over packed prompts with grouped heads, bf16
// (the pipeline of serve_attend.cuh).
//
// A segment is one query head's 256 (or 128) rows of one sequence.  Causal rows
// stop at their diagonal tile: only the tiles that some row sees are read, and
// the first 128 rows skip the last tile that only the second 128 see.  The grid
// has a block for each segment, those of a sequence from its last rows (most
// keys) to its first; a running CTA takes over blocks that have not started
// (cluster launch control), so that the next segment's copies and first
// products run under the present one's output, and the hardware's order still
// balances the SMs.
//
// Bound by the tensor cores and, beside them, by the softmax chain of the two
// streams; short prompts by the tiles of 128 that they do not fill and by the
// few segments there are.  Measured (causal): 16384 rows of 32 heads over 8 1.33
// ms, 1650 TFLOP/s; of 8 over 2 353 us, 1556; 8 x 2048 rows 222 us, 1239; 8 x 512
// 32 us, 544; 40 x 300 of 24 over 8 75 us, 296; one of 500 10.6 us.
#include "serve_attend.cuh"

namespace h3kv {
namespace serve {
namespace {

using PromptSegs = SegRing<2>;

// The register split here: the softmax warps keep the segment's bookkeeping
// beside a tile's 128 scores (at 184 they spill), the others need little.
constexpr uint32_t kRegRows = 208, kRegZero = 40, kRegCopy = 56;
static_assert(2 * kRegRows + kRegZero + kRegCopy == 512, "register split");

struct PromptSmem : Smem {
  PromptSegs segs;
  alignas(16) uint64_t taken[2];  // answer of a request for another block
  uint64_t taken_bar;
  uint64_t last_copies;           // the segment's last copies are under way
};
constexpr int kPromptSmemBytes = sizeof(PromptSmem) + 1024;
static_assert(kPromptSmemBytes <= 232448, "shared memory budget");

// Asks for a block of this grid that has not started; the answer (16 bytes)
// arrives in shared memory and counts on `bar`.  One thread.
__device__ __forceinline__ void request_block(uint32_t answer, uint32_t bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(bar)
               : "memory");
}
// The block that was taken over, or false: none is left.
__device__ __forceinline__ bool read_block(uint32_t answer, uint32_t *block) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  *block = x;
  return got != 0;
}

__device__ __forceinline__ bool counts_ok(const PromptArgs &a, int64_t q0, int64_t q1, int64_t k0, int64_t k1) {
  return q0 >= 0 && q1 >= q0 && q1 <= a.q_rows && k0 >= 0 && k1 >= k0 && k1 <= a.k_rows;
}

// Finds the segment of a block: 32 sequences at a time, going on from where
// the block before it was found (blocks mostly come in rising order).
struct Finder {
  int base = 0;        // first of the 32 sequences at hand
  int64_t before = 0;  // row tiles before them
  __device__ bool find(const PromptArgs &a, int tile_rows, uint32_t block, Seg *out) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = block / static_cast<uint32_t>(a.q_heads);
    if (unit < before) {
      base = 0;
      before = 0;
    }
    for (; base < a.seqs; base += 32) {
      const int i = base + lane;
      int64_t q0 = 0, q1 = 0, k0 = 0, k1 = 0, tiles = 0;
      if (i < a.seqs) {
        q0 = __ldg(a.cu_q + i), q1 = __ldg(a.cu_q + i + 1), k0 = __ldg(a.cu_k + i), k1 = __ldg(a.cu_k + i + 1);
        if (counts_ok(a, q0, q1, k0, k1)) tiles = (q1 - q0 + tile_rows - 1) / tile_rows;
      }
      int64_t inc = tiles;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, x);
        if (lane >= x) inc += o;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, unit < before + inc);
      if (here == 0) {
        before += __shfl_sync(0xffffffffu, inc, 31);
        continue;
      }
      const int src = __ffs(here) - 1;
      // the last rows first
      const int64_t tile = before + __shfl_sync(0xffffffffu, inc, src) - 1 - unit;
      q0 = __shfl_sync(0xffffffffu, q0, src);
      q1 = __shfl_sync(0xffffffffu, q1, src);
      k0 = __shfl_sync(0xffffffffu, k0, src);
      k1 = __shfl_sync(0xffffffffu, k1, src);
      Seg s;
      s.head = static_cast<int>(block - static_cast<uint32_t>(unit) * a.q_heads);
      s.row0 = static_cast<int>(tile * tile_rows);
      const int64_t left = q1 - q0 - s.row0;
      s.rows = static_cast<int>(left < tile_rows ? left : tile_rows);
      s.two = s.rows > kBM;
      s.keys = k1 - k0;
      s.q_base = q0;
      s.k_base = k0;
      s.diff = a.causal ? s.keys - (q1 - q0) : s.keys;
      s.nodes = 0;
      s.t0 = 0;
      s.whole = 1;
      auto tiles_of = [&](int64_t last_row) {  // key tiles that the rows up to last_row see
        int64_t see = a.causal ? last_row + s.diff + 1 : s.keys;
        see = see < 0 ? 0 : see > s.keys ? s.keys : see;
        return static_cast<int>((see + kBN - 1) / kBN);
      };
      s.n = tiles_of(s.row0 + s.rows - 1);
      s.n0 = s.two ? tiles_of(s.row0 + kBM - 1) : s.n;
      *out = s;
      return true;
    }
    return false;
  }
};

// The last tile holds rows behind the sequence's last key.
__device__ __forceinline__ bool is_ragged(const Seg &s) { return static_cast<int64_t>(s.n) * kBN > s.keys; }

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PromptArgs a, const int tile_rows) {
  extern __shared__ uint8_t smem_raw[];
  PromptSmem &sm = *reinterpret_cast<PromptSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    init_seg_ring(sm.segs, 14);
    mbar_init(smem_u32(&sm.taken_bar), 1);
    mbar_init(smem_u32(&sm.last_copies), 1);
    init_barriers(sm, false);
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  if (blockIdx.x == 0) {
    for (int i = tid; i < a.seqs; i += kThreads)
      if (!counts_ok(a, __ldg(a.cu_q + i), __ldg(a.cu_q + i + 1), __ldg(a.cu_k + i), __ldg(a.cu_k + i + 1)))
        atomicOr(a.err, kErrIndex);  // a sequence that is left out
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const WaitCtx w{a.err, &sm.abort, a.timeout_ns};
  const WaitCtx long_wait{a.err, &sm.abort, a.segment_timeout_ns};  // for the end of a segment
  SegReader<PromptSegs> sr;

  if (warp < 8) {
    // =================================================== softmax warpgroups
    reg_alloc<kRegRows>();
    const int q = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + q * 128, tO = tmem + lane_base + 256 + q * 128;
    const float c2 = a.scale_log2;
    const int i = tid & 127;  // row in the tile == TMEM lane
    uint32_t phase = 0;
    StreamEnd fin;
    while (sr.get(sm.segs, w)) {
      const Seg &s = sr.seg(sm.segs);
      if (s.rows == 0) break;
      const int r = (s.two ? q * kBM : 0) + i;  // row in the segment
      const bool warp_on = (s.two ? q * kBM : 0) + (warp & 3) * 32 < s.rows;
      // keys u < see_keys are seen by this row
      int32_t see_keys;
      {
        int64_t x = a.causal ? s.row0 + r + s.diff + 1 : s.keys;
        x = x > s.keys ? s.keys : x;
        see_keys = x < 0 ? 0 : static_cast<int32_t>(x);
      }
      Row row{kNoMax, 0.f};
      bool ok = true;
      const int step = tile_step(s), end = end_tile(s, q), t_first = first_tile(s, q);
      for (int t = t_first; t < end; t += step) {
        if (!warp_wait(smem_u32(&sm.s_full[q]), phase, w)) {
          ok = false;
          break;
        }
        phase ^= 1u;
        tc_fence_after();
        if (warp_on) {
          const int32_t n = see_keys - t * kBN;
          uint32_t see[4];
          if (__any_sync(0xffffffffu, n < kBN)) {
            prefix_mask(n, see);
            mask_tile(tS, see);
          }
          softmax_tile<false>(tS, tO, t == t_first, c2, row);
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
        const bool any = t_first < end;
        const bool none = row.l == 0.f;  // the row sees no key
        const float inv = none ? 0.f : 1.f / row.l;
        const int64_t at = s.q_base + s.row0 + r;
        uint16_t *dst = a.o.data + s.head * a.o.head_stride + at * a.o.row_stride;
        const bool live = r < s.rows;
        // a thread writes its row, 32 bytes at a time where the alignment
        // allows; a loop, since instructions that run once a segment are
        // waited for
        const float gx = ga * inv, gy = gb * inv;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          float x[16];
          if (any) {
            tmem_ld16(tO + c * 16, *reinterpret_cast<uint32_t(*)[16]>(x));
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] *= gx;
            if (joined) {
              float y[16];
              tmem_ld16(tO + 128 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(y));
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = fmaf(y[k], gy, x[k]);
            }
          }
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) h[k] = none ? 0u : pack_bf16x2(x[2 * k], x[2 * k + 1]);
          if (live) {
            if constexpr (kWide) {
              st_global_v8(dst + 16 * c, h);
            } else {
              reinterpret_cast<uint4 *>(dst)[2 * c] = make_uint4(h[0], h[1], h[2], h[3]);
              reinterpret_cast<uint4 *>(dst)[2 * c + 1] = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
        }
        if (a.lse && live)
          a.lse[s.head * a.q_rows + at] = none ? -INFINITY : kLn2 * (row.m * c2 + log2f(row.l));
      }
      fin.read_done(sm, joined);
      sr.done(sm.segs);
    }
  } else if (warp < 12) {
    // Zero the V rows behind a sequence in its last tile: P is 0 there, and 0
    // times another sequence's infinity or NaN is not.
    reg_dealloc<kRegZero>();
    Ring<kNV> vr;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && (ok = sr.get(sm.segs, long_wait))) {
      const Seg &s = sr.seg(sm.segs);
      const int n = s.n, rows = s.rows;
      const bool ragged = is_ragged(s);
      const int valid = static_cast<int>(s.keys - static_cast<int64_t>(n - 1) * kBN);
      sr.done(sm.segs);
      if (rows == 0) break;
      for (int t = 0; t < n; ++t) {
        if (ragged && t == n - 1) {
          if (!(ok = warp_wait(smem_u32(&sm.v_tail), phase, long_wait))) break;
          phase ^= 1u;
          const int r = (warp - 8) * 32 + lane;
          if (r >= valid) {
#pragma unroll
            for (int g = 0; g < 16; ++g)
              *reinterpret_cast<uint4 *>(sm.v[vr.slot] + (g >> 3) * kChunkBytes + r * 128 + (g & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.v_fixed));
        }
        vr.next();
      }
    }
  } else {
    reg_dealloc<kRegCopy>();
    if (warp == 12) {
      // ========================================================== producer
      const uint32_t go = elect_one();
      int k_issued[kNK] = {}, v_issued[kNV] = {}, q_issued[2] = {};
      uint32_t q_phase[2] = {0, 0};
      if (go) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
      }
      Ring<kNK> kr;
      Ring<kNV> vr;
      bool ok = true;
      while (ok && (ok = sr.get(sm.segs, w))) {
        const Seg s = sr.seg(sm.segs);
        sr.done(sm.segs);
        if (s.rows == 0) break;
        const int hk = s.head / a.group;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (!ok || !has_tiles(s, q)) continue;
          if (!(ok = warp_wait(smem_u32(&sm.q_free[q]), q_phase[q] ^ 1u, w))) continue;
          q_phase[q] ^= 1u;
          ++q_issued[q];
          if (go) {
            const uint32_t bar = smem_u32(&sm.q_full[q]);
            mbar_arrive_expect_tx(bar, kTileBytes);
            for (int c = 0; c < 2; ++c)
              tma_load_3d(smem_u32(sm.q[q] + c * kChunkBytes), &tm_q, c * 64,
                          static_cast<int32_t>(s.q_base + s.row0 + (s.two ? q * kBM : 0)), s.head, bar);
          }
        }
        for (int t = 0; ok && t < s.n; ++t) {
          const int32_t row = static_cast<int32_t>(s.k_base + static_cast<int64_t>(t) * kBN);
          if (!(ok = warp_wait(smem_u32(&sm.k_free[kr.slot]), kr.phase ^ 1u, w))) break;
          if (go) {
            const uint32_t bar = smem_u32(&sm.k_load[kr.slot]);
            mbar_arrive_expect_tx(bar, kTileBytes);
            tma_load_3d(smem_u32(sm.k[kr.slot]), &tm_k, 0, row, hk, bar);
            tma_load_3d(smem_u32(sm.k[kr.slot] + kChunkBytes), &tm_k, 64, row, hk, bar);
          }
          ++k_issued[kr.slot];
          kr.next();
          if (!(ok = warp_wait(smem_u32(&sm.v_free[vr.slot]), vr.phase ^ 1u, w))) break;
          if (go) {
            const uint32_t bar = smem_u32(&sm.v_load[vr.slot]);
            mbar_arrive_expect_tx(bar, kTileBytes);
            tma_load_3d(smem_u32(sm.v[vr.slot]), &tm_v, 0, row, hk, bar);
            tma_load_3d(smem_u32(sm.v[vr.slot] + kChunkBytes), &tm_v, 64, row, hk, bar);
          }
          ++v_issued[vr.slot];
          vr.next();
        }
        if (ok && go) mbar_arrive(smem_u32(&sm.last_copies));
        __syncwarp();
      }
      // every copy this thread issued must land before the CTA exits, also
      // where another warp gives up behind the last of them
      for (int q = 0; q < 2; ++q)
        if (q_issued[q]) mbar_wait_drain(smem_u32(&sm.q_full[q]), (q_issued[q] - 1) & 1, kDrainNs);
      for (int x = 0; x < kNK; ++x)
        if (k_issued[x]) mbar_wait_drain(smem_u32(&sm.k_load[x]), (k_issued[x] - 1) & 1, kDrainNs);
      for (int x = 0; x < kNV; ++x)
        if (v_issued[x]) mbar_wait_drain(smem_u32(&sm.v_load[x]), (v_issued[x] - 1) & 1, kDrainNs);
    } else if (warp == 13) {
      // ====================================================== MMA issuer
      MmaState m;
      mma_setup(m, sm, true);
      while (sr.get(sm.segs, w)) {
        const Seg s = sr.seg(sm.segs);
        sr.done(sm.segs);
        if (s.rows == 0) break;
        if (s.n > 0 && !mma_segment<false>(m, sm, s, is_ragged(s), w)) break;
      }
      // every MMA issued must finish before TMEM is released
      mma_commit(m.go, smem_u32(&sm.drain));
      mbar_wait_drain(smem_u32(&sm.drain), 0, kDrainNs);
    } else if (warp == 15) {
      // ======================================================== segments
      // a segment of no rows is the end
      Finder f;
      Ring<PromptSegs::kDepth> r;
      uint32_t block = blockIdx.x, phase = 0, copies_phase = 0;
      bool more = true;
      auto next_block = [&] {
        if (lane == 0) request_block(smem_u32(sm.taken), smem_u32(&sm.taken_bar));
        const bool came = warp_wait(smem_u32(&sm.taken_bar), phase, w);
        // (the answer must have landed before the CTA exits)
        if (!came) mbar_wait_drain(smem_u32(&sm.taken_bar), phase, kDrainNs);
        phase ^= 1u;
        const bool got = came && read_block(smem_u32(sm.taken), &block);
        // it has been read before the next one is written over it
        fence_proxy_async_smem();
        __syncwarp();
        return got;
      };
      for (;;) {
        Seg s;
        bool found = false;
        while (more && !(found = f.find(a, tile_rows, block, &s))) {
          more = next_block();  // (a block that no sequence needs)
        }
        if (!found) s.rows = s.n = 0;
        if (!warp_wait(smem_u32(&sm.segs.empty[r.slot]), r.phase ^ 1u, long_wait)) break;
        if (lane == 0) {
          sm.segs.seg[r.slot] = s;
          mbar_arrive(smem_u32(&sm.segs.full[r.slot]));
        }
        __syncwarp();
        if (!found) break;
        r.next();
        // another block is asked for only when this segment's last copies are
        // under way (two tiles before its end): taken earlier, it would wait
        // here while other SMs run out of work
        if (!warp_wait(smem_u32(&sm.last_copies), copies_phase, long_wait)) break;
        copies_phase ^= 1u;
        more = next_block();
      }
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

}  // namespace
}  // namespace serve

cudaError_t launch_attend_prompt(const PromptArgs &a, cudaStream_t stream) {
  using namespace serve;
  // whole 32-byte sectors per store where the output's alignment allows
  const bool wide = ((reinterpret_cast<uintptr_t>(a.o.data) | static_cast<uintptr_t>(a.o.head_stride * 2) |
                      static_cast<uintptr_t>(a.o.row_stride * 2)) &
                     31) == 0;
  auto kernel = wide ? prompt_kernel<true> : prompt_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  const cudaError_t e = allow_smem(kernel, kPromptSmemBytes, allowed[wide]);
  if (e != cudaSuccess) return e;
  // every sequence may end in a part of a row tile
  auto units = [&](int64_t rows) { return ((a.q_rows + rows - 1) / rows + a.seqs) * a.q_heads; };
  const int tile_rows = units(256) < 2 * a.num_sms ? 128 : 256;
  const int64_t grid = units(tile_rows);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  CUtensorMap tq, tk, tv;
  if (!encode_rows_bf16(&tq, a.q, a.q_heads, a.q_rows, 128)) return cudaErrorInvalidValue;
  tk = tv = tq;  // no keys at all: never read
  if (a.k_rows > 0 && (!encode_rows_bf16(&tk, a.k, a.kv_heads, a.k_rows, 128) ||
                       !encode_rows_bf16(&tv, a.v, a.kv_heads, a.k_rows, 128)))
    return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(grid), kThreads, kPromptSmemBytes, stream>>>(tq, tk, tv, a, tile_rows);
  return cudaGetLastError();
}

}  // namespace h3kv
