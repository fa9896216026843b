// attend_prompt.cu -- attention over packed prompts with grouped heads, bf16
// (the pipeline of serve_attend.cuh).
//
// A CTA owns one query head's 256 (or 128) rows of one sequence.  Causal rows
// stop at their diagonal tile: only the tiles that some row sees are read, and
// the first 128 rows skip the last tile that only the second 128 see.  Within
// a sequence the rows with most keys are launched first, so that the short
// CTAs fill the end.
#include "serve_attend.cuh"

namespace h3kv {
namespace serve {
namespace {

// The segment of CTA `unit` (row tiles of all sequences, each from its last to
// its first): found by a scan over the sequences.  False: nothing to do.
__device__ bool prompt_segment(const PromptArgs &a, Smem &sm, int tile_rows, Seg *out) {
  const uint32_t unit = blockIdx.x / static_cast<uint32_t>(a.q_heads);
  const int head = static_cast<int>(blockIdx.x - unit * a.q_heads);
  const int tid = threadIdx.x;
  if (tid == 0) sm.scan_seq = -1;
  int64_t before = 0;
  for (int base = 0; base < a.seqs; base += kThreads) {
    const int i = base + tid;
    int64_t tiles = 0;
    if (i < a.seqs) {
      const int64_t q0 = __ldg(a.cu_q + i), q1 = __ldg(a.cu_q + i + 1), k0 = __ldg(a.cu_k + i),
                    k1 = __ldg(a.cu_k + i + 1);
      if (q0 < 0 || q1 < q0 || q1 > a.q_rows || k0 < 0 || k1 < k0 || k1 > a.k_rows) {
        if (blockIdx.x == 0) atomicOr(a.err, kErrIndex);  // a sequence that is left out
      } else {
        tiles = (q1 - q0 + tile_rows - 1) / tile_rows;
      }
    }
    int64_t all;
    const int64_t mine = before + block_prefix(sm, tiles, &all);
    if (unit >= mine && unit < mine + tiles) {
      sm.scan_seq = i;
      sm.scan_prefix = mine + tiles - 1 - unit;  // last rows first
    }
    before += all;
    // the first CTA checks every sequence
    if (blockIdx.x != 0 && unit < before) break;
  }
  __syncthreads();
  const int i = sm.scan_seq;
  if (i < 0) return false;
  const int64_t q0 = __ldg(a.cu_q + i), q1 = __ldg(a.cu_q + i + 1), k0 = __ldg(a.cu_k + i), k1 = __ldg(a.cu_k + i + 1);
  Seg s;
  s.seq = i;
  s.head = head;
  s.row0 = static_cast<int>(sm.scan_prefix * tile_rows);
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

__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PromptArgs a, const int tile_rows) {
  extern __shared__ uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Seg s;
  if (!prompt_segment(a, sm, tile_rows, &s)) return;

  if (tid == 0) init_barriers(sm, false);
  if (warp == 13) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const WaitCtx w{a.err, &sm.abort, a.timeout_ns};
  // the last tile holds rows behind the sequence's last key
  const bool ragged = static_cast<int64_t>(s.n) * kBN > s.keys;

  if (warp < 8) {
    reg_alloc<kRegSoftmax>();
    const int q = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + q * 128, tO = tmem + lane_base + 256 + q * 128;
    const float c2 = a.scale_log2;
    const int i = tid & 127;                       // row in the tile == TMEM lane
    const int r = (s.two ? q * kBM : 0) + i;       // row in the segment
    const bool warp_on = (s.two ? q * kBM : 0) + (warp & 3) * 32 < s.rows;
    // keys u < see are seen by this row
    int64_t see_keys = a.causal ? s.row0 + r + s.diff + 1 : s.keys;
    see_keys = see_keys > s.keys ? s.keys : see_keys;
    Row row{kNoMax, 0.f};
    bool ok = true;
    uint32_t phase = 0;
    const int step = tile_step(s), end = end_tile(s, q), t_first = first_tile(s, q);
    for (int t = t_first; t < end; t += step) {
      if (!warp_wait(smem_u32(&sm.s_full[q]), phase, w)) {
        ok = false;
        break;
      }
      phase ^= 1u;
      tc_fence_after();
      if (warp_on) {
        const int64_t n = see_keys - static_cast<int64_t>(t) * kBN;
        uint32_t see[4];
        if (__any_sync(0xffffffffu, n < kBN)) {
          prefix_mask(n, see);
          softmax_tile<false, true>(tS, tO, t == t_first, see, c2, row);
        } else {
          softmax_tile<false, false>(tS, tO, t == t_first, see, c2, row);
        }
      }
      tc_fence_before();
      __syncwarp();
      // (a diagnostic may withhold one tile's arrival: see withhold_p_tile1)
      if (lane == 0 && t + 1 != a.withhold_p_tile1) mbar_arrive(smem_u32(&sm.p_full[q]));
    }
    if (s.n > 0) ok = ok && warp_wait(smem_u32(&sm.o_full), 0, w);
    tc_fence_after();
    // stream 1's maxima and sums for the join; both warpgroups leave together
    if (!s.two && q == 1) join_ml(sm)[i] = make_float2(row.m, row.l);
    ok = named_bar_and(1, 256, ok);
    if (ok && (s.two || q == 0)) {
      const bool joined = !s.two && s.n > 1;
      float ga = 1.f, gb = 0.f;
      if (joined) join_rows(row, join_ml(sm)[i], c2, ga, gb);
      const float inv = row.l == 0.f ? 0.f : 1.f / row.l;
      if (warp_on) {
        // the row as bf16 into the Q tile (free now), 16-byte granule g of
        // row i at g ^ (i mod 16), then out two rows at a time
        uint8_t *stage = sm.q[q] + i * 256;
        if (has_tiles(s, q)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x[32];
            tmem_ld32(tO + c * 32, *reinterpret_cast<uint32_t(*)[32]>(x));
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] *= ga * inv;
            if (joined) {
              float y[32];
              tmem_ld32(tO + 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(y));
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = fmaf(y[k], gb * inv, x[k]);
            }
            if (row.l == 0.f) {
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4 *>(stage + (((4 * c + k) ^ (i & 15)) << 4)) =
                  make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]), pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                             pack_bf16x2(x[8 * k + 4], x[8 * k + 5]), pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
          }
        } else {
#pragma unroll
          for (int g = 0; g < 16; ++g) *reinterpret_cast<uint4 *>(stage + g * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
        const int w0 = (warp & 3) * 32, base = s.two ? q * kBM : 0;
#pragma unroll 4
        for (int rr = 0; rr < 32; rr += 2) {
          const int ti = w0 + rr + (lane >> 4), g = lane & 15;
          if (base + ti < s.rows) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sm.q[q] + ti * 256 + ((g ^ (ti & 15)) << 4));
            *reinterpret_cast<uint4 *>(a.o.data + s.head * a.o.head_stride +
                                       (s.q_base + s.row0 + base + ti) * a.o.row_stride + g * 8) = v;
          }
        }
        if (a.lse && r < s.rows)
          a.lse[s.head * a.q_rows + s.q_base + s.row0 + r] =
              row.l == 0.f ? -INFINITY : kLn2 * (row.m * c2 + log2f(row.l));
      }
    }
  } else if (warp < 12) {
    reg_dealloc<kRegDequant>();
    // zero the V rows behind the sequence in its last tile: P is 0 there, and
    // 0 times another sequence's infinity or NaN is not
    if (ragged) {
      const int slot = (s.n - 1) % kNV;
      if (warp_wait(smem_u32(&sm.v_tail), 0, w)) {
        const int valid = static_cast<int>(s.keys - static_cast<int64_t>(s.n - 1) * kBN);
        const int r = (warp - 8) * 32 + lane;
        if (r >= valid) {
#pragma unroll
          for (int g = 0; g < 16; ++g)
            *reinterpret_cast<uint4 *>(sm.v[slot] + (g >> 3) * kChunkBytes + r * 128 + (g & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.v_fixed));
      }
    }
  } else {
    reg_dealloc<kRegIssue>();
    if (warp == 12) {
      const uint32_t go = elect_one();
      int k_issued[kNK] = {0, 0, 0}, v_issued[kNV] = {0, 0}, q_issued[2] = {0, 0};
      bool tail_issued = false;
      if (go) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (!has_tiles(s, q)) continue;
        q_issued[q] = 1;
        if (go) {
          const uint32_t bar = smem_u32(&sm.q_full[q]);
          mbar_arrive_expect_tx(bar, kTileBytes);
          for (int c = 0; c < 2; ++c)
            tma_load_3d(smem_u32(sm.q[q] + c * kChunkBytes), &tm_q, c * 64,
                        static_cast<int32_t>(s.q_base + s.row0 + (s.two ? q * kBM : 0)), s.head, bar);
        }
      }
      Ring<kNK> kr;
      Ring<kNV> vr;
      const int hk = s.head / a.group;
      for (int t = 0; t < s.n; ++t) {
        const int32_t row = static_cast<int32_t>(s.k_base + static_cast<int64_t>(t) * kBN);
        if (!warp_wait(smem_u32(&sm.k_free[kr.slot]), kr.phase ^ 1u, w)) break;
        if (go) {
          const uint32_t bar = smem_u32(&sm.k_load[kr.slot]);
          mbar_arrive_expect_tx(bar, kTileBytes);
          tma_load_3d(smem_u32(sm.k[kr.slot]), &tm_k, 0, row, hk, bar);
          tma_load_3d(smem_u32(sm.k[kr.slot] + kChunkBytes), &tm_k, 64, row, hk, bar);
        }
        ++k_issued[kr.slot];
        kr.next();
        if (!warp_wait(smem_u32(&sm.v_free[vr.slot]), vr.phase ^ 1u, w)) break;
        const bool tail = ragged && t == s.n - 1;
        if (go) {
          const uint32_t bar = tail ? smem_u32(&sm.v_tail) : smem_u32(&sm.v_load[vr.slot]);
          mbar_arrive_expect_tx(bar, kTileBytes);
          tma_load_3d(smem_u32(sm.v[vr.slot]), &tm_v, 0, row, hk, bar);
          tma_load_3d(smem_u32(sm.v[vr.slot] + kChunkBytes), &tm_v, 64, row, hk, bar);
        }
        if (tail) tail_issued = true;
        else ++v_issued[vr.slot];
        vr.next();
      }
      if (sm.abort) {
        // every copy this thread issued must land before the CTA exits
        for (int q = 0; q < 2; ++q)
          if (q_issued[q]) mbar_wait_drain(smem_u32(&sm.q_full[q]), 0, kDrainNs);
        if (tail_issued) mbar_wait_drain(smem_u32(&sm.v_tail), 0, kDrainNs);
        for (int x = 0; x < kNK; ++x)
          if (k_issued[x]) mbar_wait_drain(smem_u32(&sm.k_load[x]), (k_issued[x] - 1) & 1, kDrainNs);
        for (int x = 0; x < kNV; ++x)
          if (v_issued[x]) mbar_wait_drain(smem_u32(&sm.v_load[x]), (v_issued[x] - 1) & 1, kDrainNs);
      }
    } else if (warp == 13) {
      MmaState m;
      mma_setup(m, sm, true);
      if (s.n > 0) mma_segment<false>(m, sm, s, ragged, w);
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

}  // namespace
}  // namespace serve

cudaError_t launch_attend_prompt(const PromptArgs &a, cudaStream_t stream) {
  using namespace serve;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
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
  prompt_kernel<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(tq, tk, tv, a, tile_rows);
  return cudaGetLastError();
}

}  // namespace h3kv
