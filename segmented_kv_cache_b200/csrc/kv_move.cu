// Move cache rows between slots: what a request accepted of its drafted tokens
// goes from the draft slots to the end of its own run.
//
// A row is kv_heads * head_dim values in each pool.  One CTA per group of moves
// (and per slice of 128 columns of 16 bytes): a thread owns one 16-byte column of
// K or V and walks the group's moves eight at a time, all eight loads before the
// first store.  No move reads what an earlier one wrote, so the order inside
// the eight does not matter, and a row that an earlier move reads and a later one
// writes is read first.
#include <cuda_runtime.h>
#include <stdint.h>

#include "seg_attn_internal.h"
#include "seg_draft.h"

namespace segattn {

__device__ int g_move_error;  // non-zero once a slot out of range was skipped

namespace {

constexpr int kMoveThreads = 128;
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(
    uint4* k_pool, uint4* v_pool, const int32_t* __restrict__ src,
    const int32_t* __restrict__ dst, int64_t n_moves, const int32_t* __restrict__ offsets,
    int row_vecs, int64_t num_slots) {
  int64_t lo = blockIdx.x, hi = lo + 1;
  if (offsets) {
    lo = max((int64_t)__ldg(offsets + blockIdx.x), (int64_t)0);
    hi = min((int64_t)__ldg(offsets + blockIdx.x + 1), n_moves);
  }
  const int col = blockIdx.y * kMoveThreads + threadIdx.x;  // K columns, then V columns
  const bool live = col < 2 * row_vecs;
  uint4* pool = col < row_vecs ? k_pool + col : v_pool + (col - row_vecs);
  for (int64_t i0 = lo; i0 < hi; i0 += kBatch) {
    uint4 v[kBatch];
    int32_t d[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      d[e] = -1;
      if (i0 + e >= hi) continue;
      const int32_t a = __ldg(src + i0 + e), b = __ldg(dst + i0 + e);
      if (a == b) continue;
      if (a < 0 || a >= num_slots || b < 0 || b >= num_slots) {
        if (col == 0) atomicOr(&g_move_error, 1);
        continue;
      }
      d[e] = b;
      if (live) v[e] = pool[(int64_t)a * row_vecs];
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (live && d[e] >= 0) pool[(int64_t)d[e] * row_vecs] = v[e];
  }
}

}  // namespace

int take_move_error(int* value) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_move_error, sizeof(int)) != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_move_error, &zero, sizeof(int)) != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  *value = v;
  return SEG_ATTN_OK;
}

}  // namespace segattn

extern "C" int seg_attn_kv_move(void* k_pool, void* v_pool, const int32_t* src, const int32_t* dst,
                                int64_t n_moves, const int32_t* offsets, int64_t n_groups,
                                int kv_heads, int head_dim, int elem_bytes, int64_t num_slots,
                                void* stream) {
  if (n_moves < 0 || (offsets && n_groups < 0) || kv_heads <= 0 || head_dim <= 0 ||
      num_slots < 0 || (elem_bytes != 1 && elem_bytes != 2))
    return SEG_ATTN_ERR_INVALID_ARG;
  const int64_t row_bytes = (int64_t)kv_heads * head_dim * elem_bytes;
  if (row_bytes % 16 != 0 || row_bytes > (1 << 26)) return SEG_ATTN_ERR_UNSUPPORTED;
  const int64_t groups = offsets ? n_groups : n_moves;
  if (n_moves > INT32_MAX || groups > INT32_MAX) return SEG_ATTN_ERR_UNSUPPORTED;
  if (n_moves == 0 || groups == 0) return SEG_ATTN_OK;
  auto aligned = [](const void* p, uintptr_t a) {
    return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
  };
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(src, 4) || !aligned(dst, 4) ||
      (offsets && !aligned(offsets, 4)))
    return SEG_ATTN_ERR_INVALID_ARG;
  const int row_vecs = (int)(row_bytes / 16);
  const int slices = (2 * row_vecs + segattn::kMoveThreads - 1) / segattn::kMoveThreads;
  if (slices > 65535) return SEG_ATTN_ERR_UNSUPPORTED;
  segattn::kv_move_kernel<<<dim3((unsigned)groups, slices), segattn::kMoveThreads, 0,
                            static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), src, dst, n_moves, offsets,
      row_vecs, num_slots);
  return cudaGetLastError() == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
}
