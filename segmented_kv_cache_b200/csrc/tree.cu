// Attention of drafted tokens over the segmentable KV cache.
//
// Row (drafted token i, query head h) sees the request's P cached keys and the few
// drafted keys of its mask.  The cached keys are seen by every row alike, so the
// prefill kernel runs over them with all the request's drafted tokens packed into
// its query tiles (no mask; each K/V byte serves every token and head of the
// group) and leaves, per piece j of the key range, a normalised partial O_j and
// lse_j = log2 of its sum of exponentials.  The kernel below joins them with the
// drafted keys: both kinds are entries (score, value) of one softmax,
//   O = sum_e 2^(s_e - M) v_e / sum_e 2^(s_e - M),   lse = M + log2 sum_e 2^(s_e - M)
// with (lse_j, O_j) for a piece and (scale log2e <q, k>, v) for a drafted key (the
// per-block partials + per-request reduction of the FlashAccel article, "data
// layout optimisation").
//
// A token of a tree sees its ancestors, a handful of the drafted keys, so they
// are read one by one (the set bits of its mask row) in fp32 on the CUDA cores:
// dense tensor-core tiles would do T^2 products for T * depth useful ones, and a
// masked key's infinite or NaN value times a zero weight would reach the row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "ptx_sm100.cuh"
#include "seg_attn_internal.h"
#include "seg_draft.h"

namespace segattn {
namespace {

struct JoinParams {
  const __nv_bfloat16* q;
  const void* k_pool;
  const void* v_pool;
  __nv_bfloat16* out;
  float* lse;
  const int32_t* table;
  const int4* rows;            // [total_q][2]
  const int32_t* draft_slot;   // [total_q]
  const int4* citem;           // [items]
  const float* part_o;         // [slot][kItemRows][D]
  const float* part_lse;       // [slot][kItemRows]
  const float* k_scale;        // E4M3 pools: [kv_heads]
  const float* v_scale;
  float scale_log2;
  int q_heads, kv_heads, group;
};

__device__ __forceinline__ void bf16x2_to_f32(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two_codes, float& lo, float& hi) {
  const uint32_t h = ptx::e4m3x2_to_f16x2(two_codes);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  lo = f.x;
  hi = f.y;
}

// One warp per (drafted token, query head); four groups of eight lanes take the
// entries in turn, each lane D / 8 columns of the row, and the groups' online
// softmax states are merged at the end.  Columns of lane l of a group: bf16 rows
// 8 l .. 8 l + 7 of each 64-column half (a group's 16-byte loads are 128
// consecutive bytes), E4M3 rows D / 8 consecutive ones.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) tree_join_kernel(const JoinParams p) {
  constexpr int NC = D / 8;        // columns per lane
  constexpr int kSpan = FP8 ? NC : 8;  // consecutive columns of a lane
  const int head = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, gi = lane >> 3, l8 = lane & 7;
  if (head >= p.q_heads) return;
  const int64_t tok = blockIdx.x;
  const int4 r0 = __ldg(p.rows + 2 * tok), r1 = __ldg(p.rows + 2 * tok + 1);
  const int g = head / p.group, hh = head - g * p.group;
  // column of element j of this lane
  auto col = [&](int j) { return (j / kSpan) * 64 + l8 * kSpan + j % kSpan; };
  float q[NC], acc[NC];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < NC; ++j) acc[j] = 0.f;
  {
    const float s = FP8 ? p.scale_log2 * __ldg(p.k_scale + g) : p.scale_log2;
    const __nv_bfloat16* qr = p.q + (tok * p.q_heads + head) * D;
#pragma unroll
    for (int j = 0; j < NC; j += 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(qr + col(j));
      bf16x2_to_f32(w.x, q[j], q[j + 1]);
      bf16x2_to_f32(w.y, q[j + 2], q[j + 3]);
      bf16x2_to_f32(w.z, q[j + 4], q[j + 5]);
      bf16x2_to_f32(w.w, q[j + 6], q[j + 7]);
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) q[j] *= s;
  }
  // a lane's columns of one cache row
  auto load_row = [&](const void* pool, int32_t slot, float (&x)[NC]) {
    const int64_t row = ((int64_t)slot * p.kv_heads + g) * D;
    if constexpr (FP8) {
      const uint8_t* src = static_cast<const uint8_t*>(pool) + row + l8 * NC;
      uint32_t w[NC / 4];
      if constexpr (NC == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        w[0] = v.x, w[1] = v.y;
      }
#pragma unroll
      for (int j = 0; j < NC / 4; ++j) {
        e4m3x2_to_f32(w[j] & 0xffffu, x[4 * j], x[4 * j + 1]);
        e4m3x2_to_f32(w[j] >> 16, x[4 * j + 2], x[4 * j + 3]);
      }
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(pool) + row;
#pragma unroll
      for (int j = 0; j < NC; j += 8) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + col(j)));
        bf16x2_to_f32(w.x, x[j], x[j + 1]);
        bf16x2_to_f32(w.y, x[j + 2], x[j + 3]);
        bf16x2_to_f32(w.z, x[j + 4], x[j + 5]);
        bf16x2_to_f32(w.w, x[j + 6], x[j + 7]);
      }
    }
  };
  // add an entry: score s (log2 domain), value x, weighted by vs (1 or the V scale)
  auto add = [&](float s, const float (&x)[NC], float vs) {
    const float m_new = fmaxf(m, s);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ptx::ex2(m - base), w = ptx::ex2(s - base);
    m = m_new;
    l = l * alpha + w;
    const float wv = w * vs;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[j] = fmaf(acc[j], alpha, wv * x[j]);
  };

  // ---- the drafted keys this token sees
  const uint32_t* mask =
      reinterpret_cast<const uint32_t*>(p.table) +
      (int64_t)((uint64_t)(uint32_t)r0.z | ((uint64_t)(uint32_t)r0.w << 32));
  const float vs = FP8 ? __ldg(p.v_scale + g) : 1.f;
  for (int w = 0; w < r0.y; ++w) {
    uint32_t bits = __ldg(mask + w);
    while (bits) {
      int mine = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int b = __ffs(bits) - 1;  // -1 once no bit is left
        if (gi == e) mine = b;
        bits &= bits - 1;
      }
      float x[NC], dot = 0.f;
      float v[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) x[j] = v[j] = 0.f;
      if (mine >= 0) {
        const int32_t slot = __ldg(p.draft_slot + r0.x + 32 * w + mine);
        load_row(p.k_pool, slot, x);
        load_row(p.v_pool, slot, v);
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) dot = fmaf(q[j], x[j], dot);
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      add(mine >= 0 ? dot : -INFINITY, v, vs);
    }
  }

  // ---- the pieces over the cached keys
  if (r1.x >= 0) {
    const int4 ci = __ldg(p.citem + r1.x + g);
    for (int j = gi; j < ci.y; j += 4) {
      const int64_t prow = (int64_t)(ci.x + j) * kItemRows + r1.y + hh;
      const float* po = p.part_o + prow * D;
      float x[NC];
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 f = *reinterpret_cast<const float4*>(po + col(c));
        x[c] = f.x, x[c + 1] = f.y, x[c + 2] = f.z, x[c + 3] = f.w;
      }
      add(p.part_lse[prow], x, 1.f);
    }
  }

  // ---- merge the four groups; each lane ends with NC / 4 columns of the row
  float M = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
  const float Mb = M == -INFINITY ? 0.f : M;
  const float f = ptx::ex2(m - Mb);
  l *= f;
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
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
  __nv_bfloat16* orow = p.out + (tok * p.q_heads + head) * D + col(j0);
#pragma unroll
  for (int j = 0; j < NC / 4; j += 2)
    *reinterpret_cast<__nv_bfloat162*>(orow + j) = __floats2bfloat162_rn(o[j] * inv, o[j + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[tok * p.q_heads + head] =
        l == 0.f ? -INFINITY : (Mb + log2f(l)) * 0.69314718055994531f;
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
  if (pass.num_work > 0) {
    PrefillLaunch a;
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.out = nullptr;  // every piece writes to the workspace
    a.lse = nullptr;
    a.tab = make_view(dev_table, pass);
    a.desc = &pass;
    a.scale = softmax_scale;
    a.part_o = part_o;
    a.part_lse = part_lse;
    a.fp8 = fp8;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    const int rc = launch_prefill(a, st);
    if (rc != SEG_ATTN_OK) return rc;
  }
  const int32_t* t = static_cast<const int32_t*>(dev_table);
  JoinParams j;
  j.q = static_cast<const __nv_bfloat16*>(q);
  j.k_pool = k_pool;
  j.v_pool = v_pool;
  j.out = static_cast<__nv_bfloat16*>(out);
  j.lse = lse;
  j.table = t;
  j.rows = reinterpret_cast<const int4*>(t + desc->off_row);
  j.draft_slot = t + desc->off_draft_slot;
  j.citem = reinterpret_cast<const int4*>(t + desc->off_citem);
  j.part_o = part_o;
  j.part_lse = part_lse;
  j.k_scale = k_scale;
  j.v_scale = v_scale;
  j.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
  j.q_heads = pass.q_heads;
  j.kv_heads = pass.kv_heads;
  j.group = pass.q_heads / pass.kv_heads;
  const dim3 grid((unsigned)pass.total_q, (unsigned)((pass.q_heads + 7) / 8));
  if (grid.y > 65535) return SEG_ATTN_ERR_UNSUPPORTED;
  if (fp8) {
    if (pass.head_dim == 128)
      tree_join_kernel<128, true><<<grid, 256, 0, st>>>(j);
    else
      tree_join_kernel<64, true><<<grid, 256, 0, st>>>(j);
  } else {
    if (pass.head_dim == 128)
      tree_join_kernel<128, false><<<grid, 256, 0, st>>>(j);
    else
      tree_join_kernel<64, false><<<grid, 256, 0, st>>>(j);
  }
  return cudaGetLastError() == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
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
