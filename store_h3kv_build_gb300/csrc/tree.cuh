// tree.cuh -- what the two kernels of h3kv_attend_tree and their join share: how
// the work is listed and split over the CTAs, the workspace, a node's mask.
//
// The work is the list of all (sequence, kv head, row tile, 128-key tile)
// units in that order.  One CTA per SM takes an equal run of it, whatever the
// lengths: a segment is the part of a run that belongs to one (sequence, head,
// row tile).  A segment that holds every key tile of its rows writes the
// output; the others write their un-normalised output with (max, sum) to the
// workspace, and a second kernel joins each row's parts in order.  A CTA has at
// most two such parts: the end of an item begun before its run, and the
// beginning of one that goes on behind it.
#pragma once

#include "serve_attend.cuh"

namespace h3kv {
namespace serve {
namespace {

constexpr int kMaxCtas = 152;

// Rows of an item (a row tile of one sequence and kv head): 256 on the tcgen05
// pipeline, 8, 16 or 32 on the few-row kernel.
constexpr int kManyRows = 256;

// Which of them, by the mean rows of a sequence and kv head (the host does not
// know the single counts; every kernel is right for all of them).  Measured at
// 32 x 8192, 1 x 32768 and 128 x 1024 cached tokens, 8 kv heads, 4 query heads
// each: 8 rows 95, 20 and 62 us in items of 8, 123, 24 and 83 in items of 16; 16
// rows 124, 26 and 87 us in items of 16, 176, 30 and 111 in two of 8; 32 rows
// 161, 37 and 128 us in items of 32, 234, 38 and 162 in two of 16, 236, 43 and
// 215 on the pipeline; 40 rows 239, 43 and 221 us on the pipeline, 342, 50 and
// 235 in three items of 16 (and two of 32 would take twice the 161).
inline int item_rows_of(int32_t group, int64_t nodes, int32_t seqs) {
  const int64_t mean = (group * nodes + seqs - 1) / (seqs > 0 ? seqs : 1);
  return mean <= 8 ? 8 : mean <= 16 ? 16 : mean <= 32 ? 32 : kManyRows;
}

// An item that lies on several CTAs, as the second of them describes it to the
// join.
struct Split {
  int64_t q_base;
  int32_t parts;  // CTAs that hold its tiles, from the one before on; 0: none
  int32_t head, row0, rows;
  int32_t pad[2];
};

// Workspace: a Split per CTA, then per CTA and part un-normalised O
// [rows][128] and (max, sum) [rows].
struct Workspace {
  Split *split;
  float *o;
  float2 *ml;
  int rows;  // rows of a part
};
__host__ __device__ inline int part_rows(int group, int64_t nodes, int item_rows) {
  const int64_t n = group * (nodes < H3KV_TREE_MAX_NODES ? nodes : H3KV_TREE_MAX_NODES);
  return n < item_rows ? static_cast<int>(n) : item_rows;
}
__device__ inline Workspace workspace_of(const TreeArgs &a) {
  Workspace ws;
  uint8_t *p = reinterpret_cast<uint8_t *>(a.workspace);
  ws.rows = part_rows(a.group, a.nodes, a.item_rows);
  ws.split = reinterpret_cast<Split *>(p);
  ws.o = reinterpret_cast<float *>(p + kMaxCtas * sizeof(Split));
  ws.ml = reinterpret_cast<float2 *>(ws.o + static_cast<int64_t>(a.ctas) * 2 * ws.rows * 128);
  return ws;
}

// What an item costs beside its key tiles (query rows, first page, output, join),
// in tiles: its first units, to which no tile belongs.  Sequences of very
// different lengths tell: 33 of 64 .. 32768 cached rows, 32 heads over 8, took 91,
// 80, 80 and 83 us at 2, 3, 4 and 6 tiles (one token each: items of 8 rows), 139,
// 118, 104 and 106 (4 nodes: items of 16), and 243, 218 and 220 us at 4, 6 and 8
// (64 nodes).  100 of 64 .. 8192: 102, 86, 88 and 93; 161, 129, 116 and 121; 278,
// 268 and 280.  Items of 32 (8 nodes) at 4, 5 and 7: 154, 142 and 145; 170, 159 and
// 162.
inline int item_cost_of(int32_t item_rows) { return item_rows == kManyRows ? 6 : item_rows == 32 ? 5 : item_rows == 16 ? 4 : 3; }

// A sequence's counts; tiles == 0: nothing to do (empty, or out of range).
struct Counts {
  int64_t q_base;
  int32_t len, nodes, tiles, row_tiles;
  int64_t units;
  bool bad;
};
__device__ __forceinline__ Counts counts_of(const TreeArgs &a, int i) {
  const int64_t c0 = __ldg(a.cu_nodes + i), c1 = __ldg(a.cu_nodes + i + 1), len = __ldg(a.lengths + i), m = c1 - c0;
  Counts c;
  c.bad = c0 < 0 || m < 0 || c1 > a.nodes || m > H3KV_TREE_MAX_NODES || len < m ||
          len > (a.max_pages << a.p.page_shift) || len > INT32_MAX - 256;
  const bool on = !c.bad && m > 0;
  c.q_base = c0;
  c.len = on ? static_cast<int32_t>(len) : 0;
  c.nodes = on ? static_cast<int32_t>(m) : 0;
  c.tiles = (c.len + kBN - 1) / kBN;
  c.row_tiles = (c.nodes * a.group + a.item_rows - 1) >> (31 - __clz(a.item_rows));  // 0 without nodes
  c.units = static_cast<int64_t>(c.tiles + a.item_cost) * c.row_tiles * a.p.kv_heads;
  return c;
}

// CTAs that get work, each at least one unit, and the first unit of one.
__device__ __forceinline__ int working(const TreeArgs &a, int64_t total) {
  return total < a.ctas ? static_cast<int>(total) : a.ctas;
}
__device__ __forceinline__ int64_t first_unit(int64_t total, int cta, int ctas) { return total * cta / ctas; }
// The CTA that holds unit u: the last k with total k / ctas < u + 1.
__device__ __forceinline__ int owner_of(int64_t total, int64_t u, int ctas) {
  return static_cast<int>(((u + 1) * ctas - 1) / total);
}

// This CTA's run of units: found by all threads of the block, kept in shared
// memory (scratch: 32 words there).  CTA 0 also checks every sequence.
struct Scan {
  int64_t total;
  int64_t u0, u1;
  int64_t before;  // units before sequence `seq`, which holds unit u0
  Counts c;        // of that sequence
  int seq, ctas;
};

template <int kBlock>
__device__ __forceinline__ int64_t block_prefix(int64_t *warp_sum, int64_t v, int64_t *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t inc = v;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, x);
    if (lane >= x) inc += o;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t below = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kBlock / 32; ++w) {
    const int64_t t = warp_sum[w];
    below += w < warp ? t : 0;
    all += t;
  }
  *total = all;
  return below + inc - v;
}

template <int kBlock>
__device__ __forceinline__ void find_run(const TreeArgs &a, Scan &sc, int64_t *scratch) {
  const int tid = threadIdx.x;
  int64_t total = 0;
  int64_t at = 0;  // units before this thread's sequence
  Counts c = {};
  for (int base = 0; base < a.seqs; base += kBlock) {
    const int i = base + tid;
    int64_t all;
    c = {};
    if (i < a.seqs) {
      c = counts_of(a, i);
      if (c.bad && blockIdx.x == 0) atomicOr(a.p.err, kErrIndex);
    }
    at = total + block_prefix<kBlock>(scratch, c.units, &all);
    total += all;
  }
  const int ctas = working(a, total), cta = static_cast<int>(blockIdx.x);
  const int64_t u0 = cta < ctas ? first_unit(total, cta, ctas) : total;
  const int64_t u1 = cta < ctas ? first_unit(total, cta + 1, ctas) : total;
  if (tid == 0) {
    sc.total = total;
    sc.u0 = u0;
    sc.u1 = u1;
    sc.ctas = ctas;
  }
  // the sequence that holds u0: known already where one round covered them all
  int64_t before = 0;
  for (int base = 0; base < a.seqs && u0 < u1; base += kBlock) {
    if (a.seqs > kBlock) {
      const int i = base + tid;
      int64_t all;
      c = {};
      if (i < a.seqs) c = counts_of(a, i);
      at = before + block_prefix<kBlock>(scratch, c.units, &all);
      before += all;
    }
    if (c.units > 0 && u0 >= at && u0 < at + c.units) {
      sc.seq = base + tid;
      sc.before = at;
      sc.c = c;
    }
    if (a.seqs > kBlock && u0 < before) break;
  }
  __syncthreads();
}

// The segments of a run of units, one after the other.
struct Walk {
  int64_t u, end;     // units left: [u, end)
  int64_t before;     // units before sequence `seq`
  int seq;
  Counts c;
  __device__ __forceinline__ void start(const TreeArgs &a, const Scan &sc) {
    u = sc.u0;
    end = sc.u1;
    seq = sc.seq;
    before = sc.before;
    c = sc.c;
  }
  __device__ __forceinline__ bool next(const TreeArgs &a, Seg *s) {
    while (u < end) {
      while (u >= before + c.units) {
        before += c.units;
        c = counts_of(a, ++seq);
      }
      const int size = c.tiles + a.item_cost;
      const int64_t w = u - before, item = w / size;
      const int off = static_cast<int>(w - item * size);
      const int take = end - u < size - off ? static_cast<int>(end - u) : size - off;
      u += take;
      const int t0 = off > a.item_cost ? off - a.item_cost : 0, t1 = off + take - a.item_cost;
      if (t1 <= t0) continue;
      s->t0 = t0;
      s->n = s->n0 = t1 - t0;
      s->head = static_cast<int>(item / c.row_tiles);
      s->row0 = static_cast<int>(item - static_cast<int64_t>(s->head) * c.row_tiles) * a.item_rows;
      const int rows = c.nodes * a.group - s->row0;
      s->rows = rows < a.item_rows ? rows : a.item_rows;
      s->two = s->rows > kBM;
      s->keys = c.len;
      s->q_base = c.q_base;
      s->k_base = static_cast<int64_t>(seq) * a.max_pages;
      s->nodes = c.nodes;
      s->seq = seq;
      s->diff = 0;
      s->whole = s->n == c.tiles;
      return true;
    }
    s->n = 0;
    return false;
  }
};

using TreeSegs = SegRing<2>;
using TreeReader = SegReader<TreeSegs>;

// Describes the item that the CTA's run goes on with, where it began on the CTA
// before, to the join.
__device__ __forceinline__ Split split_of(const TreeArgs &a, const Scan &sc) {
  Split split = {};
  const int size = sc.c.tiles + a.item_cost, cta = static_cast<int>(blockIdx.x);
  const int64_t item = (sc.u0 - sc.before) / size;
  // its tiles' units
  const int64_t first = sc.before + item * size + a.item_cost, last = first + sc.c.tiles - 1;
  if (sc.u0 > first && owner_of(sc.total, first, sc.ctas) == cta - 1) {
    split.q_base = sc.c.q_base;
    split.parts = owner_of(sc.total, last, sc.ctas) - cta + 2;
    split.head = static_cast<int>(item / sc.c.row_tiles);
    split.row0 = static_cast<int>(item - static_cast<int64_t>(split.head) * sc.c.row_tiles) * a.item_rows;
    const int rows = sc.c.nodes * a.group - split.row0;
    split.rows = rows < a.item_rows ? rows : a.item_rows;
  }
  return split;
}

// The walking warp.  (The others wait for the first segment: it goes out before
// anything else is done.)  `then` is called behind each segment that went out,
// with its slot, and says whether to go on.
template <class Then>
__device__ __forceinline__ void publish_segments(const TreeArgs &a, const Scan &sc, const Workspace &ws,
                                                 TreeSegs &ring, const WaitCtx &w, const Then &then) {
  Walk walk;
  walk.start(a, sc);
  Ring<TreeSegs::kDepth> r;
  bool described = false;
  const WaitCtx long_wait{w.err, w.abort, a.segment_timeout_ns};  // a slot falls free when its segment is done
  for (;;) {
    Seg s;
    const bool more = walk.next(a, &s);
    if (!warp_wait(smem_u32(&ring.empty[r.slot]), r.phase ^ 1u, long_wait)) return;
    if ((threadIdx.x & 31) == 0) {
      ring.seg[r.slot] = s;
      mbar_arrive(smem_u32(&ring.full[r.slot]));
    }
    __syncwarp();
    const bool go = more && then(s, r.slot);
    if (!described) {
      described = true;
      const Split split = split_of(a, sc);
      if ((threadIdx.x & 31) == 0) ws.split[blockIdx.x] = split;
    }
    if (!go) return;
    r.next();
  }
}
// The node of row x of a sequence and kv head: x / group by a multiply and a
// shift, exact for x below 64 * 64 (the error is below 2^-7, group at most 64).
__device__ __forceinline__ int node_of(const TreeArgs &a, int x) {
  return static_cast<int>((static_cast<uint32_t>(x) * a.group_magic) >> 19);
}

// Node j's path to its root as bits.
__device__ __forceinline__ uint64_t path_of(const TreeArgs &a, int64_t q_base, int j) {
  if (!a.parents) return (2ull << j) - 1;
  uint64_t path = 0;
  for (int n = j; n >= 0;) {
    path |= 1ull << n;
    const int up = __ldg(a.parents + q_base + n);
    n = up >= 0 && up < n ? up : -1;
  }
  return path;
}

// The 128-column mask of a row for the tile at key `pos`: all keys below
// `base`, and node i's key base + i where bit i of `path` is set.
__device__ __forceinline__ void tree_mask(int32_t pos, int32_t base, uint64_t path, uint32_t (&see)[4]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int32_t off = base - (pos + 32 * g);  // columns below off come before the nodes
    if (off >= 32) see[g] = 0xffffffffu;
    else if (off >= 0) see[g] = ((1u << off) - 1u) | static_cast<uint32_t>(path << off);
    else see[g] = off > -64 ? static_cast<uint32_t>(path >> -off) : 0u;
  }
}

// The page of the row at token `pos`; a page out of range is reported and
// page 0 read in its place.
__device__ __forceinline__ int32_t page_at(const TreeArgs &a, int64_t table, int32_t pos) {
  const int32_t page = __ldg(a.page_table + table + (pos >> a.p.page_shift));
  if (page < 0 || page >= a.p.pages) {
    atomicOr(a.p.err, kErrIndex);
    return 0;
  }
  return page;
}

}  // namespace
}  // namespace serve
}  // namespace h3kv
