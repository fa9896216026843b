// serve_attend.cuh -- the attention pipeline of the serving operators on sm_103a
// tensor cores (tcgen05 + TMEM): packed prompts over bf16 K/V, and trees of
// drafted tokens over the paged kvi8r cache.
//
// A CTA works through segments: up to 256 query rows that share one kv head,
// over a run of 128-key tiles.  Two softmax warpgroups (thread = row = TMEM
// lane) keep two score tiles in flight, so that one's softmax overlaps the
// other's matrix products:
//   rows > 128 ("two"):  warpgroup q owns rows 128 q .. 128 q + 127 and sees
//                        every key tile;
//   rows <= 128:         both own the same rows, warpgroup q sees the key tiles
//                        of parity q, and the two running softmaxes are joined
//                        by their log-sum-exp at the segment's end.
// So few rows keep both halves of the pipeline busy too, and their keys are
// read once.  (Trees of up to 32 rows a sequence and kv head have a kernel of
// their own.)
//
// Warp roles (512 threads):
//   warps 0-3, 4-7  softmax, correction and epilogue of stream 0 / 1
//   warps 8-11      cache: in-place int8 -> fp16 dequantisation of K and V
//                   tiles, query rows of later segments; prompts: zeroing of
//                   the V rows behind a sequence
//   warp 12         prompts: TMA copies of Q, K and V; cache: bulk copies of
//                   K's codes
//   warp 13         TMEM allocation and tcgen05.mma issue
//   warp 14         cache: bulk copies of V's codes; prompts: idle
//   warp 15         finds the segments
// TMEM (512 columns, fp32): S0 [0,128), S1 [128,256), P over the first 64
// columns of its S, O0 [256,384), O1 [384,512).
#pragma once

#include <math.h>

#include "attend.cuh"
#include "serve_rows.cuh"

namespace h3kv {
namespace serve {

using attn::kBM;
using attn::kBN;
using attn::kChunkBytes;
using attn::kLazyRescaleLog2;
using attn::kNK;
using attn::kNV;
using attn::kThreads;
using attn::kTileBytes;
using attn::warp_wait;

// Register split per warpgroup, sums to 512 = 4 x 128 (the launch's share).
constexpr uint32_t kRegSoftmax = 184, kRegDequant = 80, kRegIssue = 64;
static_assert(2 * kRegSoftmax + kRegDequant + kRegIssue == 512, "register split");

// "No key yet" in a running maximum.  (Not a low finite value: bf16 operands
// reach any score that fp32 holds.)
constexpr float kNoMax = -INFINITY;
// Up to this |maximum| of a tile in log2 units a weight is ex2(s c2 - m c2) with
// m c2 rounded to fp32: the rounding, at most 2^-9, is common to the weights
// that are relative to m.  Beyond, where it would grow to whole powers of two,
// m is subtracted from the scores before the product.
constexpr float kFusedMaxLog2 = 65536.f;

// fp16 weights carry a factor of 2^7: relative to a maximum that may have grown
// by 2^8 they stay below 2^15, and what fp16 cannot hold lies below 2^-32 of the
// maximum (an error of 2^-12 over a million keys; 2^-5 without the factor, where
// weights of 2^-25 were lost).  bf16 weights need none.
constexpr float kWeightLog2 = 7.f, kWeightInv = 0.0078125f;

struct Smem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kNK][kTileBytes];
  uint8_t v[kNV][kTileBytes];
  float2 ml[kBM];  // stream 1's (max, sum) for the join with stream 0
  uint64_t q_full[2];
  uint64_t k_load[kNK], k_ready[kNK], k_free[kNK];
  uint64_t v_load[kNV], v_ready[kNV], v_free[kNV];
  uint64_t s_full[2], p_full[2];
  uint64_t o_full[2], drain;
  uint64_t ml_full[4], ml_free[4];  // per warp: stream 1's ml are written; its O and ml have been read
  uint64_t q_free[2];        // the stream's last QK of a segment is done
  uint64_t v_tail, v_fixed;  // prompts: a ragged last V tile has come; its rest is zeroed
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

// Ring slot and phase, advanced tile by tile over all segments.
template <int kDepth>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kDepth) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// One segment: key tiles t0 .. t0 + n - 1 of a sequence for up to 256 rows.
struct Seg {
  int n;          // key tiles that any row sees
  int n0;         // ... that stream 0's rows see (two: n0 <= n; else n)
  int t0;
  int two;
  int rows;
  int row0;       // first row in the sequence's row numbering
  int head;       // prompt: query head; cache: kv head
  int64_t keys;   // keys of the sequence
  int64_t q_base; // first row of the sequence in Q
  int64_t k_base; // prompt: first row of the sequence in K; cache: its first page table entry
  int64_t diff;   // prompt, causal: row t sees the keys u <= t + diff
  int nodes;      // cache: drafted nodes
  int seq;        // cache: not read; without it ptxas allots the few-row kernel's
                  // registers otherwise, and items of 32 rows (8 nodes of four
                  // heads over 32 x 8192 rows) took 169 us in place of 161
  int whole;      // every key tile of the rows is in this segment
};

// Tiles of stream q in a segment: first, step and end.
__device__ __forceinline__ int first_tile(const Seg &s, int q) { return s.two ? 0 : q; }
__device__ __forceinline__ int tile_step(const Seg &s) { return s.two ? 1 : 2; }
__device__ __forceinline__ int end_tile(const Seg &s, int q) { return s.two && q == 0 ? s.n0 : s.n; }
__device__ __forceinline__ bool has_tiles(const Seg &s, int q) { return first_tile(s, q) < end_tile(s, q); }

// The segments go through a short ring in shared memory: one warp finds
// them (its 64-bit divisions and counts would otherwise take registers and
// instruction cache in every role), the others read.  A segment of no tiles is the end.
template <int kSegs>
struct SegRing {
  static constexpr int kDepth = kSegs;
  Seg seg[kDepth];
  uint64_t full[kDepth], empty[kDepth];
};
template <int kSegs>
__device__ __forceinline__ void init_seg_ring(SegRing<kSegs> &r, int readers) {
  for (int i = 0; i < kSegs; ++i) {
    mbar_init(smem_u32(&r.full[i]), 1);
    mbar_init(smem_u32(&r.empty[i]), readers);
  }
}
// A reading warp: get() waits for the next segment, done() lets it go.
template <class Segs>
struct SegReader {
  Ring<Segs::kDepth> r;
  __device__ __forceinline__ bool get(Segs &ring, const WaitCtx &w) {
    return warp_wait(smem_u32(&ring.full[r.slot]), r.phase, w);
  }
  __device__ __forceinline__ const Seg &seg(const Segs &ring) const { return ring.seg[r.slot]; }
  __device__ __forceinline__ void done(Segs &ring) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ring.empty[r.slot]));
    r.next();
  }
};

__device__ __forceinline__ void init_barriers(Smem &sm, bool cache) {
  for (int q = 0; q < 2; ++q) {
    mbar_init(smem_u32(&sm.q_full[q]), cache ? 4 : 1);
    mbar_init(smem_u32(&sm.s_full[q]), 1);
    mbar_init(smem_u32(&sm.o_full[q]), 1);
    mbar_init(smem_u32(&sm.q_free[q]), 1);
    mbar_init(smem_u32(&sm.p_full[q]), 4);
  }
  for (int s = 0; s < kNK; ++s) {
    mbar_init(smem_u32(&sm.k_load[s]), 1);
    mbar_init(smem_u32(&sm.k_ready[s]), 4);
    mbar_init(smem_u32(&sm.k_free[s]), 1);
  }
  for (int s = 0; s < kNV; ++s) {
    mbar_init(smem_u32(&sm.v_load[s]), 1);
    mbar_init(smem_u32(&sm.v_ready[s]), 4);
    mbar_init(smem_u32(&sm.v_free[s]), 1);
  }
  for (int i = 0; i < 4; ++i) {
    mbar_init(smem_u32(&sm.ml_full[i]), 1);
    mbar_init(smem_u32(&sm.ml_free[i]), 1);
  }
  mbar_init(smem_u32(&sm.drain), 1);
  mbar_init(smem_u32(&sm.v_tail), 1);
  mbar_init(smem_u32(&sm.v_fixed), 4);
  sm.abort = 0;
  fence_mbar_init();
}

// ------------------------------------------------------------- MMA issuer --
// The warp runs this converged; one elected lane issues.  Order per key tile
// and stream: PV of the tile, then QK of the stream's next tile, so that the
// completion of a QK also covers the PV before it.
struct MmaState {
  uint32_t go, tmem, dhi, lq0, lk0, lv0, idesc_qk, idesc_pv;
  Ring<kNK> k;        // the next key tile whose QK is to be issued first
  Ring<kNV> v;
  uint32_t p_phase = 0, q_phase = 0;  // bit q: of stream q
  uint32_t fix_phase = 0;
};

__device__ __forceinline__ void mma_setup(MmaState &m, Smem &sm, bool bf16) {
  m.go = elect_one();
  m.tmem = sm.tmem_base;
  m.idesc_qk = idesc_f16(bf16, false, kBM, kBN);
  m.idesc_pv = idesc_f16(bf16, true, kBM, 128);
  const uint64_t dq0 = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024);
  m.dhi = static_cast<uint32_t>(dq0 >> 32);
  m.lq0 = static_cast<uint32_t>(dq0);
  m.lk0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(sm.k[0]), 16, 1024));
  m.lv0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(sm.v[0]), kChunkBytes, 1024));
}

__device__ __forceinline__ void issue_qk(const MmaState &m, uint32_t tS, uint32_t lq, uint32_t lk) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
    mma_ss(m.go, tS, lq + off, lk + off, m.dhi, m.idesc_qk, kk > 0);
  }
}

__device__ __forceinline__ void issue_pv(const MmaState &m, uint32_t tS, uint32_t lv, uint32_t acc) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(m.go, tS + 256, tS + kk * 8, lv + (kk * 2048 >> 4), m.dhi, m.idesc_pv,
           (acc || kk > 0) ? 1u : 0u);
}

// One segment's products.  kReady: tiles are handed over by the dequantising
// warps (k_ready, v_ready); otherwise by the copies (k_load, v_load), and a
// ragged last V tile goes through the warps that zero its rest (v_tail,
// v_fixed).  A stream's Q tile is let go (q_free) after its last QK, so that
// the next segment's rows come in under this one's end.
template <bool kReady>
__device__ __forceinline__ bool mma_segment(MmaState &m, Smem &sm, const Seg &s, bool ragged, const WaitCtx &w) {
  uint64_t *k_rdy = kReady ? sm.k_ready : sm.k_load;
  uint64_t *v_rdy = kReady ? sm.v_ready : sm.v_load;
  // the stream's QK of tile t: waits for the tile (its first user does), and
  // releases it after its last user
  auto qk = [&](int q, uint32_t tS, uint32_t lq, uint32_t lk, bool first_user, bool last_user, bool last_qk) {
    if (first_user) {
      if (!warp_wait(smem_u32(&k_rdy[m.k.slot]), m.k.phase, w)) return false;
      tc_fence_after();
    }
    issue_qk(m, tS, lq, lk);
    mma_commit(m.go, smem_u32(&sm.s_full[q]));
    if (last_user) {
      mma_commit(m.go, smem_u32(&sm.k_free[m.k.slot]));
      m.k.next();
    }
    if (last_qk) mma_commit(m.go, smem_u32(&sm.q_free[q]));
    return true;
  };
#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    if (!has_tiles(s, q)) continue;
    if (!warp_wait(smem_u32(&sm.q_full[q]), (m.q_phase >> q) & 1u, w)) return false;
    m.q_phase ^= 1u << q;
    tc_fence_after();
    // two: both streams start on tile 0 (stream 1 alone where stream 0 has none)
    const bool first_user = !s.two || q == 0 || s.n0 == 0;
    if (!qk(q, m.tmem + q * 128, m.lq0 + q * (kTileBytes >> 4), m.lk0 + m.k.slot * (kTileBytes >> 4), first_user,
            !s.two || q == 1, first_tile(s, q) + tile_step(s) >= end_tile(s, q))) return false;
  }
  const int step = tile_step(s);
  for (int t = 0; t < s.n; ++t) {
    if (!warp_wait(smem_u32(&v_rdy[m.v.slot]), m.v.phase, w)) return false;
    if (!kReady && ragged && t == s.n - 1) {
      // (the rows' softmax of this tile still runs)
      if (m.go) mbar_arrive(smem_u32(&sm.v_tail));
      __syncwarp();
      if (!warp_wait(smem_u32(&sm.v_fixed), m.fix_phase, w)) return false;
      m.fix_phase ^= 1u;
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int q = s.two ? i : (t & 1);
      if (!s.two && i == 1) break;
      const int end = end_tile(s, q), tn = t + step;
      if (t >= end) continue;
      // everything that the products need is at hand before the wait
      uint32_t tS = m.tmem + q * 128, lv = m.lv0 + m.v.slot * (kTileBytes >> 4), lq = m.lq0 + q * (kTileBytes >> 4),
               lk = m.lk0 + m.k.slot * (kTileBytes >> 4), acc = t != first_tile(s, q);
      const bool last = !s.two || q == 1, more = tn < end, first_user = !s.two || q == 0 || tn >= s.n0;
      asm volatile("" : "+r"(tS), "+r"(lv), "+r"(lq), "+r"(lk), "+r"(acc));
      if (!warp_wait(smem_u32(&sm.p_full[q]), (m.p_phase >> q) & 1u, w)) return false;
      tc_fence_after();
      issue_pv(m, tS, lv, acc);
      m.p_phase ^= 1u << q;
      if (last) mma_commit(m.go, smem_u32(&sm.v_free[m.v.slot]));
      if (!more) {
        mma_commit(m.go, smem_u32(&sm.o_full[q]));
        continue;
      }
      if (!qk(q, tS, lq, lk, first_user, last, tn + step >= end)) return false;
    }
    m.v.next();
  }
  return true;
}

// ---------------------------------------------------------------- softmax --
struct Row {
  float m, l;  // running maximum (raw score units) and sum of this thread's row
};

// Masks a tile's scores in TMEM: only the columns set in `see` count, whatever
// the others hold.  A pass of its own, and a loop, because few tiles need it
// and the kernels' code has to stay in the instruction caches.  With the mask in
// a second copy of softmax_tile and the MMA issue unrolled over the streams, CTAs
// that were at different places of their segments pushed each other's code out:
// warps waited for instructions 2.5 cycles per issue (0.65 where all CTAs ran in
// step), and 64 nodes over 128 x 2048 cached tokens took 411 us, then 338; 40
// prompts of 300 tokens 85 us, then 76.
__device__ __forceinline__ void mask_tile(uint32_t tS, const uint32_t (&see)[4]) {
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    const uint32_t bits = g == 0 ? see[0] : g == 1 ? see[1] : g == 2 ? see[2] : see[3];
    if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
    uint32_t x[32];
    tmem_ld32(tS + 32 * g, x);
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = (bits >> c) & 1u ? x[c] : 0xff800000u;  // -infinity
    tmem_st32(tS + 32 * g, x);
  }
  tmem_wait_st();
}

// Subtracts `ref` from a tile's scores in TMEM, a loop like mask_tile.
__device__ __forceinline__ void shift_tile(uint32_t tS, float ref) {
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    uint32_t x[32];
    tmem_ld32(tS + 32 * g, x);
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) - ref);
    tmem_st32(tS + 32 * g, x);
  }
  tmem_wait_st();
}

// One 128-key tile: S from TMEM, running maximum, P back to TMEM.
template <bool kF16>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, bool first, float c2, Row &r) {
  float s[128];
  float m4[4];
  tmem_ld128_max(tS, *reinterpret_cast<uint32_t(*)[128]>(s), m4);
  const float mt = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
  if (first) {
    r.m = mt;
    r.l = 0.f;
  }
  // O is rescaled only when the maximum grows by more than 2^8 (exact: the
  // weights are relative to r.m, whatever it is); infinite differences from and
  // to kNoMax give a factor of 0 and no growth.  The two rare cases share one
  // vote: with a vote of its own for `far`, 40 prompts of 300 tokens took 87 us,
  // 79 so and without.
  const bool need = (mt - r.m) * c2 > kLazyRescaleLog2, far = fabsf(mt) * c2 > kFusedMaxLog2 && mt != kNoMax;
  float cm = c2;
  if (__any_sync(0xffffffffu, need || far)) {
    if (!first) {
      const float alpha = need ? ex2((r.m - mt) * c2) : 1.f;
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
      shift_tile(tS, r.m == kNoMax ? 0.f : r.m);
      tmem_ld128_max(tS, *reinterpret_cast<uint32_t(*)[128]>(s), m4);
      cm = 0.f;
    }
  }
  constexpr float kUp = kF16 ? kWeightLog2 : 0.f;
  const float bias = r.m == kNoMax ? kUp : fmaf(-r.m, cm, kUp);  // (kNoMax: all scores are -infinity)
  const float2 cc = make_float2(c2, c2), nm = make_float2(bias, bias);
  float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int c = h * 64 + 2 * k;
      float2 e = __ffma2_rn(make_float2(s[c], s[c + 1]), cc, nm);
      e.x = ex2(e.x);
      e.y = ex2(e.y);
      if (k & 1) acc1 = __fadd2_rn(acc1, e);
      else acc0 = __fadd2_rn(acc0, e);
      pk[k] = attn::pack2<kF16>(e.x, e.y);
    }
    tmem_st32(tS + h * 32, pk);
  }
  tmem_wait_st();
  const float2 acc = __fadd2_rn(acc0, acc1);
  r.l += acc.x + acc.y;
}

// Columns below `n` of a 128-column tile, as bits.
__device__ __forceinline__ void prefix_mask(int32_t n, uint32_t (&see)[4]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int32_t k = n - 32 * g;
    see[g] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
  }
}

// Joins stream 1's (max, sum) into r: the weights of the two streams' O.
__device__ __forceinline__ void join_rows(Row &r, float2 other, float c2, float &ga, float &gb) {
  const float m = fmaxf(r.m, other.x), ref = m == kNoMax ? 0.f : m;
  ga = ex2((r.m - ref) * c2);
  gb = ex2((other.x - ref) * c2);
  r.l = fmaf(r.l, ga, other.y * gb);
  r.m = m;
}

// The end of a segment for a softmax warp; the warps do not wait for one
// another.  at_end waits for the stream's O.  Where the two streams share their
// rows, stream 1 hands its (max, sum) over and waits until its O has been read,
// and stream 0 takes both.  kOff: nothing to write (stream 1 of shared rows, or
// a warp without rows); kFailed: a wait ran out.
enum End { kFailed, kOff, kWrite };
struct StreamEnd {
  uint32_t o_phase[2] = {0, 0};
  uint32_t ml_phase = 0;
  __device__ __forceinline__ End at_end(Smem &sm, const Seg &s, int q, bool warp_on, Row &row, float c2, bool *joined,
                                        float *ga, float *gb, const WaitCtx &w) {
    const int wi = (threadIdx.x >> 5) & 3, i = threadIdx.x & 127;
    const bool share = !s.two && s.n > 1;
    bool ok = true;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!has_tiles(s, x)) continue;
      if (x == q || (share && q == 0)) ok = ok && warp_wait(smem_u32(&sm.o_full[x]), o_phase[x], w);
      o_phase[x] ^= 1u;
    }
    if (!ok) return kFailed;
    tc_fence_after();
    *joined = false;
    *ga = 1.f;
    *gb = 0.f;
    if (!warp_on) return kOff;
    if (s.two) return kWrite;
    if (q == 1) {
      if (!share) return kOff;
      sm.ml[i] = make_float2(row.m, row.l);
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.ml_full[wi]));
      ok = warp_wait(smem_u32(&sm.ml_free[wi]), ml_phase, w);
      ml_phase ^= 1u;
      tc_fence_after();
      return ok ? kOff : kFailed;
    }
    if (share) {
      if (!warp_wait(smem_u32(&sm.ml_full[wi]), ml_phase, w)) return kFailed;
      ml_phase ^= 1u;
      join_rows(row, sm.ml[i], c2, *ga, *gb);
      *joined = true;
    }
    return kWrite;
  }
  // The warp has read what O it needed.
  __device__ __forceinline__ void read_done(Smem &sm, bool joined) const {
    tc_fence_before();
    __syncwarp();
    if (joined && (threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.ml_free[(threadIdx.x >> 5) & 3]));
  }
};

constexpr float kLn2 = 0.6931471805599453f;

}  // namespace serve
}  // namespace h3kv
