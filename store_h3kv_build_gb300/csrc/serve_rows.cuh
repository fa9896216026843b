// serve_rows.cuh -- rows of 128 values held by 8 lanes, as the serving operators
// read, rotate and write them.
#pragma once

#include "ptx.cuh"
#include "serve.h"

namespace h3kv {

// 32 bytes from global memory; the address must be 32-byte aligned.
__device__ __forceinline__ void ld_global_v8(const void *p, uint4 &a, uint4 &b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

// 16 bytes from global to shared memory without a register; zeros where !in.
// copy16_wait: this thread's copies are done.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// TMA store of a box from shared memory, in groups of this thread's own; at
// most kPending groups may still be reading shared memory after the wait.
__device__ __forceinline__ void tma_store_3d(const void *map, uint32_t src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void bulk_wait_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void unpack_bf16x8(const uint4 w, float *x) {
  x[0] = bf16lo_to_f32(w.x);
  x[1] = bf16hi_to_f32(w.x);
  x[2] = bf16lo_to_f32(w.y);
  x[3] = bf16hi_to_f32(w.y);
  x[4] = bf16lo_to_f32(w.z);
  x[5] = bf16hi_to_f32(w.z);
  x[6] = bf16lo_to_f32(w.w);
  x[7] = bf16hi_to_f32(w.w);
}

// Unnormalised FWHT of a 128-value row held by 8 neighbouring lanes: value
// 64 hi + 8 l + e of the row is x[8 hi + e] of the group's lane l, so that a
// row's loads and stores are two runs of 8 lanes x 16 bytes.  Strides 1, 2, 4
// and 64 run in registers, strides 8, 16, 32 between lanes: 48 shuffles for
// the warp's 4 rows, against 80 with a row across the warp.  All but stride 1
// take two values an instruction (a - b as fma(b, -1, a), the same rounding).
__device__ __forceinline__ void fwht128_oct(float (&x)[16], int l) {
  const float2 neg = make_float2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float a = x[i], b = x[i + 1];
    x[i] = a + b;
    x[i + 1] = a - b;
  }
#pragma unroll
  for (int h = 2; h < 16; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      if ((i & h) == 0) {
        const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[i + h], x[i + h + 1]);
        const float2 s = __fadd2_rn(a, b), d = __ffma2_rn(b, neg, a);
        x[i] = s.x;
        x[i + 1] = s.y;
        x[i + h] = d.x;
        x[i + h + 1] = d.y;
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    const float sg = (l & m) ? -1.f : 1.f;
    const float2 sign = make_float2(sg, sg);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, x[i], m), __shfl_xor_sync(0xffffffffu, x[i + 1], m));
      const float2 z = __ffma2_rn(make_float2(x[i], x[i + 1]), sign, o);
      x[i] = z.x;
      x[i + 1] = z.y;
    }
  }
}

}  // namespace h3kv
