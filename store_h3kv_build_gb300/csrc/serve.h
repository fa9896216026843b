// serve.h -- internal launchers and device state behind h3kv_serve.h (not part
// of the public header).  The C-ABI layer has checked the arguments before any
// launcher is called; index arrays in device memory are checked by the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/h3kv_serve.h"

namespace h3kv {

// Bit of the device error word: an index array held a value out of range.
constexpr uint32_t kErrIndex = 4u;

// Current device's state, set up on the first call (abi.cu).
struct ServeDevice {
  uint32_t *err;
  int num_sms;
  uint64_t timeout_ns;
  int32_t withhold_p_tile1;  // diagnostic, see h3kv_debug_withhold_p
};
h3kv_status serve_device(ServeDevice *out);

// 3-D map over strided bf16 [heads, rows, 128]: box 64 columns x box_rows rows
// x 1 head, 128-byte swizzle; rows past `rows` read as zero (abi.cu).
bool encode_rows_bf16(CUtensorMap *m, const h3kv_rows &r, int64_t heads, int64_t rows, uint32_t box_rows);

// Allows `kernel` its dynamic shared memory, once per device (`done`: a bit for
// each of the 64 devices the library knows).
template <class Kernel>
inline cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct PagedArgs {
  int8_t *k_codes, *v_codes;
  uint16_t *k_scales, *v_scales;
  int32_t pages, kv_heads, page_size, page_shift;
  uint32_t *err;
};

cudaError_t launch_paged_append(const PagedArgs &p, const h3kv_rows &K, const h3kv_rows &V, const int32_t *rows,
                                int64_t n, const ServeDevice &d, cudaStream_t stream);
cudaError_t launch_paged_read(const PagedArgs &p, const int32_t *rows, int64_t n, const h3kv_rows &K,
                              const h3kv_rows &V, const ServeDevice &d, cudaStream_t stream);
cudaError_t launch_paged_copy(const PagedArgs &p, const int32_t *src, const int32_t *dst, int64_t n,
                              cudaStream_t stream);
cudaError_t launch_paged_keep(const PagedArgs &p, const int32_t *page_table, int64_t max_pages,
                              const int32_t *lengths, const int32_t *cu_nodes, int32_t seqs, const uint8_t *keep,
                              int64_t nodes, int32_t *new_lengths, cudaStream_t stream);

struct TreeArgs {
  PagedArgs p;
  h3kv_rows q, o;
  float *lse;
  const int32_t *page_table, *lengths, *cu_nodes, *parents;
  int64_t max_pages, nodes;
  int32_t q_heads, group, seqs;
  uint32_t group_magic;  // ceil(2^19 / group)
  float scale_log2;
  float *workspace;
  int32_t ctas;
  int32_t item_rows;   // rows of a row tile, by the kernel that runs, and
  int32_t item_cost;   //   what one costs beside its key tiles, in tiles
  uint64_t timeout_ns, segment_timeout_ns;  // of a wait, and of one for a segment's end
  int32_t withhold_p_tile1;
};
size_t tree_workspace_bytes(int32_t q_heads, int32_t kv_heads, int64_t nodes, int32_t seqs);
cudaError_t launch_attend_tree(const TreeArgs &a, cudaStream_t stream);
// Its kernel for a.item_rows 8, 16 or 32 (launch_attend_tree adds the join).
cudaError_t launch_tree_few(const TreeArgs &a, cudaStream_t stream);
// 2-D map over 8-bit codes [rows, 128]: box 128 x box_rows, 128-byte swizzle.
bool encode_codes(CUtensorMap *m, const void *base, int64_t rows, uint32_t box_rows);

struct PromptArgs {
  h3kv_rows q, k, v, o;
  float *lse;
  const int32_t *cu_q, *cu_k;
  int64_t q_rows, k_rows;
  int32_t q_heads, kv_heads, group, seqs, causal;
  float scale_log2;
  uint32_t *err;
  uint64_t timeout_ns, segment_timeout_ns;
  int32_t withhold_p_tile1;
  int32_t num_sms;
};
cudaError_t launch_attend_prompt(const PromptArgs &a, cudaStream_t stream);

}  // namespace h3kv
