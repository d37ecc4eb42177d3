// Packed forms of the calls of seg_draft.h for the Python binding: every argument in
// order as one block of 64-bit values (pointers, integers, a float as the bits of a
// double), so that a call converts one argument instead of 10 to 23.
#include <stdint.h>
#include <string.h>

#include "seg_draft.h"

namespace {

// Arguments in order.
struct Args {
  const int64_t* at;
  template <typename T>
  T* ptr() {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(*at++));
  }
  int64_t i64() { return *at++; }
  // out-of-range values must not wrap into valid ones
  int i32() {
    const int64_t v = *at++;
    return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : static_cast<int>(v);
  }
  float f32() {
    double d;
    memcpy(&d, at++, sizeof(d));
    return static_cast<float>(d);
  }
};

}  // namespace

extern "C" int seg_attn_rope_packed(const int64_t* block) {
  Args a{block};
  const void* x = a.ptr<const void>();
  const int64_t x_stride = a.i64();
  void* out = a.ptr<void>();
  const int64_t out_stride = a.i64();
  const int32_t* positions = a.ptr<const int32_t>();
  const int64_t n = a.i64();
  const int heads = a.i32(), head_dim = a.i32();
  const seg_attn_rope_desc* rope = a.ptr<const seg_attn_rope_desc>();
  const int backward = a.i32();
  return seg_attn_rope(x, x_stride, out, out_stride, positions, n, heads, head_dim, rope, backward,
                       a.ptr<void>());
}

namespace {

int append(const int64_t* block, bool fp8) {
  Args a{block};
  const void* q = a.ptr<const void>();
  const int64_t q_stride = a.i64();
  void* q_out = a.ptr<void>();
  const int64_t q_out_stride = a.i64();
  const void* k = a.ptr<const void>();
  const int64_t k_stride = a.i64();
  const void* v = a.ptr<const void>();
  const int64_t v_stride = a.i64();
  const int32_t* positions = a.ptr<const int32_t>();
  const int32_t* slots = a.ptr<const int32_t>();
  const int64_t n = a.i64();
  const int q_heads = a.i32(), kv_heads = a.i32(), head_dim = a.i32();
  const seg_attn_rope_desc* rope = a.ptr<const seg_attn_rope_desc>();
  const float* k_scale = fp8 ? a.ptr<const float>() : nullptr;
  const float* v_scale = fp8 ? a.ptr<const float>() : nullptr;
  void* k_pool = a.ptr<void>();
  void* v_pool = a.ptr<void>();
  const int64_t num_slots = a.i64();
  void* stream = a.ptr<void>();
  if (fp8)
    return seg_attn_rope_append_fp8(q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride,
                                    positions, slots, n, q_heads, kv_heads, head_dim, rope, k_scale,
                                    v_scale, k_pool, v_pool, num_slots, stream);
  return seg_attn_rope_append(q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, positions,
                              slots, n, q_heads, kv_heads, head_dim, rope, k_pool, v_pool,
                              num_slots, stream);
}

int tree(const int64_t* block, bool fp8) {
  Args a{block};
  const void* q = a.ptr<const void>();
  const void* k_pool = a.ptr<const void>();
  const void* v_pool = a.ptr<const void>();
  const float* k_scale = fp8 ? a.ptr<const float>() : nullptr;
  const float* v_scale = fp8 ? a.ptr<const float>() : nullptr;
  void* out = a.ptr<void>();
  float* lse = a.ptr<float>();
  const void* table = a.ptr<const void>();
  const seg_attn_tree_desc* desc = a.ptr<const seg_attn_tree_desc>();
  const float scale = a.f32();
  void* workspace = a.ptr<void>();
  const size_t bytes = static_cast<size_t>(a.i64());
  void* stream = a.ptr<void>();
  if (fp8)
    return seg_attn_tree_fp8(q, k_pool, v_pool, k_scale, v_scale, out, lse, table, desc, scale,
                             workspace, bytes, stream);
  return seg_attn_tree(q, k_pool, v_pool, out, lse, table, desc, scale, workspace, bytes, stream);
}

}  // namespace

extern "C" int seg_attn_rope_append_packed(const int64_t* block) { return append(block, false); }
extern "C" int seg_attn_rope_append_fp8_packed(const int64_t* block) { return append(block, true); }
extern "C" int seg_attn_tree_packed(const int64_t* block) { return tree(block, false); }
extern "C" int seg_attn_tree_fp8_packed(const int64_t* block) { return tree(block, true); }

extern "C" int seg_attn_kv_move_packed(const int64_t* block) {
  Args a{block};
  void* k_pool = a.ptr<void>();
  void* v_pool = a.ptr<void>();
  const int32_t* src = a.ptr<const int32_t>();
  const int32_t* dst = a.ptr<const int32_t>();
  const int64_t n = a.i64();
  const int32_t* offsets = a.ptr<const int32_t>();
  const int64_t groups = a.i64();
  const int kv_heads = a.i32(), head_dim = a.i32(), elem_bytes = a.i32();
  const int64_t num_slots = a.i64();
  return seg_attn_kv_move(k_pool, v_pool, src, dst, n, offsets, groups, kv_heads, head_dim,
                          elem_bytes, num_slots, a.ptr<void>());
}
