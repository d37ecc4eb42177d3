// Attention of drafted tokens over the segmentable KV cache.
//
// Row (drafted token i, query head h) sees the request's cached keys and the drafted
// keys of its mask.  The prefill kernel does it (prefill_sm100.cu, TREE): a request's
// drafted tokens x the heads of a kv head are packed into 128-row query tiles, so
// each K/V byte is read once for all of them; the K tiles that hold drafted keys take
// the mask's bits instead of the causal comparison; an item whose keys are one piece
// writes its rows itself.  An item cut along its keys leaves, per piece j, a
// normalised partial O_j and lse_j = log2 of its sum of exponentials, merged here:
//   O = sum_j 2^(lse_j - M) O_j / sum_j 2^(lse_j - M),   lse = M + log2 sum_j 2^(lse_j - M)
// (the per-block partials + per-request reduction of the FlashAccel article, "data
// layout optimisation").
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "ptx_sm100.cuh"
#include "seg_attn_internal.h"
#include "seg_draft.h"

namespace segattn {
namespace {

struct MergeParams {
  __nv_bfloat16* out;
  float* lse;
  TableView tab;
  const float* part_o;    // [slot][kItemRows][D]
  const float* part_lse;  // [slot][kItemRows]
  int q_heads, group, qpt;
};

// One warp per row of a split item.  One request's call is cut into many pieces (37 for
// 8 kv heads), so four groups of eight lanes take the pieces in turn, each lane D / 8
// columns, and the groups' online softmax states are merged at the end.  Columns of
// lane l of a group: 8 l .. 8 l + 7 of each 64-column half.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const MergeParams p) {
  constexpr int NC = D / 8;  // columns per lane
  const int4 m0 = __ldg(p.tab.merge + 2 * blockIdx.x), m1 = __ldg(p.tab.merge + 2 * blockIdx.x + 1);
  const int req = m0.x, g = m0.y, q0 = m0.z, slot0 = m0.w, parts = m1.x;
  const int tok0 = __ldg(p.tab.q_offsets + req);
  const int q_len = __ldg(p.tab.q_offsets + req + 1) - tok0;
  const int lane = threadIdx.x & 31, gi = lane >> 3, l8 = lane & 7;
  // launched as a programmatic dependent of the prefill pass, which gives no early trigger:
  // this grid starts once the pass's CTAs have exited (the launch itself is hidden), and
  // what follows reads the partials
  ptx::grid_dependency_wait();
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int qi = q0 + (row / kTileRows) * p.qpt + (row % kTileRows) / p.group;
  if (qi >= q_len) return;
  const int64_t orow = (int64_t)(tok0 + qi) * p.q_heads + g * p.group + row % p.group;
  auto col = [&](int j) { return (j >> 3) * 64 + l8 * 8 + (j & 7); };
  float acc[NC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < NC; ++j) acc[j] = 0.f;
  for (int j = gi; j < parts; j += 4) {
    const int64_t prow = (int64_t)(slot0 + j) * kItemRows + row;
    const float* po = p.part_o + prow * D;
    float x[NC];
#pragma unroll
    for (int c = 0; c < NC; c += 4) {
      const float4 f = *reinterpret_cast<const float4*>(po + col(c));
      x[c] = f.x, x[c + 1] = f.y, x[c + 2] = f.z, x[c + 3] = f.w;
    }
    const float s = p.part_lse[prow];
    const float m_new = fmaxf(m, s);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ptx::ex2(m - base), w = ptx::ex2(s - base);
    m = m_new;
    l = l * alpha + w;
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = fmaf(acc[c], alpha, w * x[c]);
  }
  float M = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
  const float Mb = M == -INFINITY ? 0.f : M;
  const float f = ptx::ex2(m - Mb);
  l *= f;
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  // sum over the groups, halving the columns a lane keeps at each step
  float h[NC / 2], o[NC / 4];
  const bool up16 = (lane & 16) != 0, up8 = (lane & 8) != 0;
#pragma unroll
  for (int j = 0; j < NC / 2; ++j) {
    const float lo = acc[j] * f, hi = acc[j + NC / 2] * f;
    const float other = __shfl_xor_sync(0xffffffffu, up16 ? lo : hi, 16);
    h[j] = (up16 ? hi : lo) + other;
  }
#pragma unroll
  for (int j = 0; j < NC / 4; ++j) {
    const float lo = h[j], hi = h[j + NC / 4];
    const float other = __shfl_xor_sync(0xffffffffu, up8 ? lo : hi, 8);
    o[j] = (up8 ? hi : lo) + other;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int j0 = (up16 ? NC / 2 : 0) + (up8 ? NC / 4 : 0);
#pragma unroll
  for (int j = 0; j < NC / 4; j += 2)
    *reinterpret_cast<__nv_bfloat162*>(p.out + orow * D + col(j0) + j) =
        __floats2bfloat162_rn(o[j] * inv, o[j + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[orow] = l == 0.f ? -INFINITY : (Mb + log2f(l)) * 0.69314718055994531f;
}

bool aligned(const void* p, uintptr_t a) {
  return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int tree(const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
         const float* v_scale, bool fp8, void* out, float* lse, const void* dev_table,
         const seg_attn_tree_desc* desc, float softmax_scale, void* workspace,
         size_t workspace_bytes, void* stream) {
  if (!desc || desc->magic != SEG_ATTN_TREE_MAGIC || desc->version != SEG_ATTN_TREE_VERSION)
    return SEG_ATTN_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return SEG_ATTN_ERR_INVALID_ARG;
  const seg_attn_table_desc& pass = desc->pass;
  if (pass.total_q == 0) return SEG_ATTN_OK;
  // a drafted token has at least its own row in the pool
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
      !aligned(dev_table, 16) || (lse && !aligned(lse, 4)))
    return SEG_ATTN_ERR_INVALID_ARG;
  if (fp8 && (!aligned(k_scale, 4) || !aligned(v_scale, 4))) return SEG_ATTN_ERR_INVALID_ARG;
  if (desc->workspace_bytes > 0 &&
      (workspace_bytes < desc->workspace_bytes || !aligned(workspace, 16)))
    return SEG_ATTN_ERR_WORKSPACE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceLayout at = workspace_layout(pass, false);
  float* part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + at.main_o);
  float* part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + at.main_lse);
  const uint32_t* words = static_cast<const uint32_t*>(dev_table);
  PrefillLaunch a;
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.out = out;
  a.lse = lse;
  a.tab = make_view(dev_table, pass);
  a.desc = &pass;
  a.scale = softmax_scale;
  a.part_o = part_o;
  a.part_lse = part_lse;
  a.fp8 = fp8;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.mask_base = words;
  a.draft_slot = reinterpret_cast<const int32_t*>(words + desc->off_draft_slot);
  const int rc = launch_prefill(a, st);
  if (rc != SEG_ATTN_OK || pass.num_merge == 0) return rc;
  MergeParams m;
  m.out = static_cast<__nv_bfloat16*>(out);
  m.lse = lse;
  m.tab = a.tab;
  m.part_o = part_o;
  m.part_lse = part_lse;
  m.q_heads = pass.q_heads;
  m.group = pass.q_heads / pass.kv_heads;
  m.qpt = pass.queries_per_tile;
  // no item has rows past the first tile when every draft fits in it
  const dim3 grid(pass.num_merge,
                  (desc->max_draft <= pass.queries_per_tile ? kTileRows : kItemRows) / 8);
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  const cudaError_t e = pass.head_dim == 128 ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<128>, m)
                                             : cudaLaunchKernelEx(&cfg, tree_merge_kernel<64>, m);
  return e == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace segattn

extern "C" int seg_attn_tree(const void* q, const void* k_pool, const void* v_pool, void* out,
                             float* lse, const void* dev_table, const seg_attn_tree_desc* desc,
                             float softmax_scale, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return segattn::tree(q, k_pool, v_pool, nullptr, nullptr, false, out, lse, dev_table, desc,
                       softmax_scale, workspace, workspace_bytes, stream);
}

extern "C" int seg_attn_tree_fp8(const void* q, const void* k_pool, const void* v_pool,
                                 const float* k_scale, const float* v_scale, void* out, float* lse,
                                 const void* dev_table, const seg_attn_tree_desc* desc,
                                 float softmax_scale, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return segattn::tree(q, k_pool, v_pool, k_scale, v_scale, true, out, lse, dev_table, desc,
                       softmax_scale, workspace, workspace_bytes, stream);
}
