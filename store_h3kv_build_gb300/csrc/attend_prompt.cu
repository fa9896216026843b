// attend_prompt.cu -- attention over packed prompts with grouped heads.
#include <math.h>

#include "ptx.cuh"
#include "serve.h"

namespace h3kv {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float dot4(const float (&a)[4], uint2 w) {
  return a[0] * bf16lo_to_f32(w.x) + a[1] * bf16hi_to_f32(w.x) + a[2] * bf16lo_to_f32(w.y) +
         a[3] * bf16hi_to_f32(w.y);
}

// One warp for a query row of one head: lane l holds values 4l .. 4l+3 of the
// row and of its running output; a key costs one dot product over the lanes
// and one step of the online softmax.
__global__ void __launch_bounds__(kWarps * 32) prompt_kernel(const PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.seqs; i += blockDim.x) {
      const int q0 = __ldg(a.cu_q + i), q1 = __ldg(a.cu_q + i + 1), k0 = __ldg(a.cu_k + i), k1 = __ldg(a.cu_k + i + 1);
      if (q0 < 0 || q1 < q0 || q1 > a.q_rows || k0 < 0 || k1 < k0 || k1 > a.k_rows) atomicOr(a.err, kErrIndex);
    }
  }
  const int64_t row = unit / a.q_heads;
  const int h = static_cast<int>(unit - row * a.q_heads);
  if (row >= a.q_rows) return;
  // the sequence whose rows hold `row`
  int lo = 0, hi = a.seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_q + mid + 1) <= row) lo = mid + 1;
    else hi = mid;
  }
  if (lo == a.seqs) return;
  const int64_t q0 = __ldg(a.cu_q + lo), q1 = __ldg(a.cu_q + lo + 1), k0 = __ldg(a.cu_k + lo),
                k1 = __ldg(a.cu_k + lo + 1);
  if (row < q0 || row >= q1) return;
  if (q0 < 0 || q1 > a.q_rows || k0 < 0 || k1 < k0 || k1 > a.k_rows) return;
  const int64_t nk = k1 - k0;
  int64_t see = a.causal ? row - q0 + 1 + nk - (q1 - q0) : nk;
  if (see < 0) see = 0;
  const uint2 qw = *reinterpret_cast<const uint2 *>(a.q.data + h * a.q.head_stride + row * a.q.row_stride + 4 * lane);
  const float q[4] = {bf16lo_to_f32(qw.x), bf16hi_to_f32(qw.x), bf16lo_to_f32(qw.y), bf16hi_to_f32(qw.y)};
  const int hk = h / a.group;
  const uint16_t *kp = a.k.data + hk * a.k.head_stride + k0 * a.k.row_stride + 4 * lane;
  const uint16_t *vp = a.v.data + hk * a.v.head_stride + k0 * a.v.row_stride + 4 * lane;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t u = 0; u < see; ++u) {
    float s = dot4(q, *reinterpret_cast<const uint2 *>(kp + u * a.k.row_stride));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float c = m == -INFINITY ? 0.f : ex2(m - mn), p = mn == -INFINITY ? 0.f : ex2(s - mn);
    const uint2 vw = *reinterpret_cast<const uint2 *>(vp + u * a.v.row_stride);
    l = l * c + p;
    o[0] = o[0] * c + p * bf16lo_to_f32(vw.x);
    o[1] = o[1] * c + p * bf16hi_to_f32(vw.x);
    o[2] = o[2] * c + p * bf16lo_to_f32(vw.y);
    o[3] = o[3] * c + p * bf16hi_to_f32(vw.y);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  *reinterpret_cast<uint2 *>(a.o.data + h * a.o.head_stride + row * a.o.row_stride + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse && lane == 0)
    a.lse[h * a.q_rows + row] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}

}  // namespace

cudaError_t launch_attend_prompt(const PromptArgs &a, cudaStream_t stream) {
  const int64_t units = a.q_rows * a.q_heads;
  prompt_kernel<<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace h3kv
