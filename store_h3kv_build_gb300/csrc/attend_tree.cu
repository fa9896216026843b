// attend_tree.cu -- attention of drafted tokens over the paged kvi8r cache.
#include <math.h>

#include "ptx.cuh"
#include "serve.h"

namespace h3kv {
namespace {

constexpr int kWarps = 8;

// One warp for a query row of one head, as a loop over the row's keys.
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const TreeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.seqs; i += blockDim.x) {
      const int64_t c0 = __ldg(a.cu_nodes + i), c1 = __ldg(a.cu_nodes + i + 1), len = __ldg(a.lengths + i);
      if (c0 < 0 || c1 < c0 || c1 > a.nodes || c1 - c0 > H3KV_TREE_MAX_NODES || len < c1 - c0 ||
          len > (a.max_pages << a.p.page_shift))
        atomicOr(a.p.err, kErrIndex);
    }
  }
  const int64_t row = unit / a.q_heads;
  const int h = static_cast<int>(unit - row * a.q_heads);
  if (row >= a.nodes) return;
  int lo = 0, hi = a.seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_nodes + mid + 1) <= row) lo = mid + 1;
    else hi = mid;
  }
  if (lo == a.seqs) return;
  const int64_t c0 = __ldg(a.cu_nodes + lo), c1 = __ldg(a.cu_nodes + lo + 1);
  const int64_t len = __ldg(a.lengths + lo), m_nodes = c1 - c0;
  if (row < c0 || row >= c1) return;
  if (c0 < 0 || c1 > a.nodes || m_nodes > H3KV_TREE_MAX_NODES || len < m_nodes ||
      len > (a.max_pages << a.p.page_shift))
    return;
  const int j = static_cast<int>(row - c0);
  uint64_t path = 0;
  for (int n = j; n >= 0;) {
    path |= 1ull << n;
    const int up = a.parents ? __ldg(a.parents + c0 + n) : n - 1;
    n = up >= 0 && up < n ? up : -1;
  }
  const uint2 qw = *reinterpret_cast<const uint2 *>(a.q.data + h * a.q.head_stride + row * a.q.row_stride + 4 * lane);
  float q[4] = {bf16lo_to_f32(qw.x), bf16hi_to_f32(qw.x), bf16lo_to_f32(qw.y), bf16hi_to_f32(qw.y)};
  fwht128_warp(q, lane);
#pragma unroll
  for (int t = 0; t < 4; ++t) q[t] = __half2float(__float2half_rn(q[t] * kInvSqrt128));
  const int hk = h / a.group;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t u = 0; u < len; ++u) {
    const int64_t node = u - (len - m_nodes);
    if (node >= 0 && !((path >> node) & 1)) continue;
    const int32_t page = __ldg(a.page_table + lo * a.max_pages + (u >> a.p.page_shift));
    if (page < 0 || page >= a.p.pages) {
      if (lane == 0) atomicOr(a.p.err, kErrIndex);
      return;
    }
    const int64_t at = ((static_cast<int64_t>(page) * a.p.kv_heads + hk) << a.p.page_shift) +
                       (u & (a.p.page_size - 1));
    const uint32_t kw = reinterpret_cast<const uint32_t *>(a.p.k_codes + at * 128)[lane];
    const uint32_t vw = reinterpret_cast<const uint32_t *>(a.p.v_codes + at * 128)[lane];
    const __half ks = __ushort_as_half(a.p.k_scales[at]), vs = __ushort_as_half(a.p.v_scales[at]);
    float s = 0.f, v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s += q[t] * __half2float(__hmul(__int2half_rn(static_cast<int8_t>(kw >> (8 * t))), ks));
      v[t] = __half2float(__hmul(__int2half_rn(static_cast<int8_t>(vw >> (8 * t))), vs));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float c = m == -INFINITY ? 0.f : ex2(m - mn), p = mn == -INFINITY ? 0.f : ex2(s - mn);
    l = l * c + p;
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = o[t] * c + p * v[t];
    m = mn;
  }
  fwht128_warp(o, lane);
  const float inv = kInvSqrt128 / l;
  *reinterpret_cast<uint2 *>(a.o.data + h * a.o.head_stride + row * a.o.row_stride + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse && lane == 0) a.lse[h * a.nodes + row] = 0.6931471805599453f * (m + log2f(l));
}

}  // namespace

size_t tree_workspace_bytes(int32_t, int32_t, int64_t, int32_t) { return 16; }

cudaError_t launch_attend_tree(const TreeArgs &a, cudaStream_t stream) {
  const int64_t units = a.nodes * a.q_heads;
  tree_kernel<<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace h3kv
