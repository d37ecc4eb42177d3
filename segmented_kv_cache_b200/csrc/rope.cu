// Rotary positions: the rotation of bf16 rows, and the append of rotated keys and
// values to the cache (the plan is made in rope_plan.cpp).
//
// Angles.  The plan holds each pair's frequency as a fraction of a turn in units
// of 2^-64, so position * frequency modulo 2^64 (one wrapping 64-bit product) is
// the angle, already reduced, for every int32 position; its upper 32 bits as a
// signed number over 2^31 are half turns in [-1, 1), which sincospif takes.  The
// error is that of one fp32 rounding (2^-24 of the half turn), far positions
// included, where fp32 position * frequency would lose every digit.
//
// Work.  Memory-bound: every value is read and written once.  A unit is 16 values
// of one head (two 16-byte vectors: with the half layout the vectors that hold the
// two sides of eight pairs).  A CTA takes a run of consecutive units, loads its
// threads' vectors first, computes the cosines and sines of the run's tokens once
// into shared memory while those loads fly, then turns and stores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "seg_attn_internal.h"
#include "seg_draft.h"

namespace segattn {

__device__ int g_rope_error;  // non-zero once a slot out of range was skipped

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnit = 16;  // values per unit

struct RopeParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* q_out;
  int64_t q_stride, q_out_stride, k_stride, v_stride;  // elements per token
  const int32_t* positions;
  const int32_t* slots;
  int64_t n_tokens, num_slots;
  void *k_pool, *v_pool;
  const float *k_scale, *v_scale;  // E4M3 pools
  int q_heads, kv_heads, head_dim, rotary;
  int head_units, token_units;     // units per head, per token
  int cta_units, cta_tokens;       // units of one CTA, and the most tokens they touch
  float amp, sign;                 // sign -1: the transposed rotation
  uint64_t turns[SEG_ATTN_ROPE_MAX_PAIRS];
};

// Cosine and sine, times the amplitude, of pair i at position pos.
__device__ __forceinline__ float2 cos_sin(uint64_t turns, int32_t pos, float amp, float sign) {
  const uint64_t angle = (uint64_t)(int64_t)pos * turns;
  const float half_turns = (float)(int32_t)(angle >> 32) * (1.f / 2147483648.f);
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(amp * c, amp * sign * s);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// E4M3 codes of eight values over the head's scale, as seg_attn_kv_append_fp8's.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned short code;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(code)
        : "f"(x[2 * i + 1] / scale), "f"(x[2 * i] / scale));
    w[i] = code;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Where a unit of the flat order (token, then query heads, key heads, value
// heads, then units of the head) lives.
struct Unit {
  int64_t token;
  int head;   // of its kind
  int kind;   // 0 query, 1 key, 2 value
  int u;      // unit of the head
};
__device__ __forceinline__ Unit locate(const RopeParams& p, int64_t t0, int at) {
  Unit x;
  const int tl = at / p.token_units;
  const int rest = at - tl * p.token_units;
  int h = rest / p.head_units;
  x.u = rest - h * p.head_units;
  x.token = t0 + tl;
  x.kind = h < p.q_heads ? 0 : h < p.q_heads + p.kv_heads ? 1 : 2;
  x.head = h - (x.kind == 0 ? 0 : x.kind == 1 ? p.q_heads : p.q_heads + p.kv_heads);
  return x;
}

// NI: units per thread and pass.  A CTA's units are a multiple of kRopeThreads * NI
// or the whole call.
template <bool INTERLEAVED, bool FP8, int NI>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  // [tokens of this CTA][8][rotary / 16]: pair 8 u + e of a token at e * (rotary / 16) + u,
  // so that the units u of neighbouring lanes read neighbouring values
  extern __shared__ float2 cs[];
  const int64_t first = (int64_t)blockIdx.x * p.cta_units;
  const int64_t total = p.n_tokens * p.token_units;
  const int count = (int)min((int64_t)p.cta_units, total - first);
  const int64_t t0 = first / p.token_units;
  const int off0 = (int)(first - t0 * p.token_units);
  const int pairs = p.rotary / 2, rot_units = p.rotary / kUnit;

  for (int base = 0; base < count; base += kRopeThreads * NI) {
    uint4 a[NI], b[NI];
    Unit un[NI];
    int32_t slot[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = base + i * kRopeThreads + threadIdx.x;
      un[i].kind = -1;
      if (at >= count) continue;
      un[i] = locate(p, t0, off0 + at);
      const Unit& x = un[i];
      const __nv_bfloat16* row =
          (x.kind == 0   ? p.q + x.token * p.q_stride
           : x.kind == 1 ? p.k + x.token * p.k_stride
                         : p.v + x.token * p.v_stride) + x.head * p.head_dim;
      const bool split = !INTERLEAVED && x.kind != 2 && x.u < rot_units;
      const int ca = split ? 8 * x.u : kUnit * x.u;
      a[i] = *reinterpret_cast<const uint4*>(row + ca);
      b[i] = *reinterpret_cast<const uint4*>(row + (split ? ca + pairs : ca + 8));
      if (x.kind != 0) slot[i] = __ldg(p.slots + x.token);
    }
    if (base == 0) {
      const int tokens = (off0 + count - 1) / p.token_units + 1;
      for (int i = threadIdx.x; i < tokens * pairs; i += kRopeThreads) {
        const int t = i / pairs, j = i - t * pairs;
        cs[t * pairs + (j & 7) * rot_units + (j >> 3)] =
            cos_sin(p.turns[j], __ldg(p.positions + t0 + t), p.amp, p.sign);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const Unit& x = un[i];
      if (x.kind < 0) continue;
      float xa[8], xb[8];
      unpack8(a[i], xa);
      unpack8(b[i], xb);
      const bool rot = x.kind != 2 && x.u < rot_units;
      const bool split = !INTERLEAVED && rot;
      if (rot) {
        const float2* c = cs + (int)(x.token - t0) * pairs + x.u;
        if (INTERLEAVED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c0 = c[e * rot_units], c1 = c[(e + 4) * rot_units];
            const float a0 = xa[2 * e], a1 = xa[2 * e + 1], b0 = xb[2 * e], b1 = xb[2 * e + 1];
            xa[2 * e] = a0 * c0.x - a1 * c0.y;
            xa[2 * e + 1] = a1 * c0.x + a0 * c0.y;
            xb[2 * e] = b0 * c1.x - b1 * c1.y;
            xb[2 * e + 1] = b1 * c1.x + b0 * c1.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 cc = c[e * rot_units];
            const float x0 = xa[e], x1 = xb[e];
            xa[e] = x0 * cc.x - x1 * cc.y;
            xb[e] = x1 * cc.x + x0 * cc.y;
          }
        }
      }
      const int ca = split ? 8 * x.u : kUnit * x.u, cb = split ? ca + pairs : ca + 8;
      if (x.kind == 0) {
        __nv_bfloat16* row = p.q_out + x.token * p.q_out_stride + x.head * p.head_dim;
        *reinterpret_cast<uint4*>(row + ca) = rot ? pack8(xa) : a[i];
        *reinterpret_cast<uint4*>(row + cb) = rot ? pack8(xb) : b[i];
        continue;
      }
      if (slot[i] < 0 || slot[i] >= p.num_slots) {
        if (x.head == 0 && x.u == 0) atomicOr(&g_rope_error, 1);
        continue;
      }
      const int64_t at = ((int64_t)slot[i] * p.kv_heads + x.head) * p.head_dim;
      void* pool = x.kind == 1 ? p.k_pool : p.v_pool;
      if (FP8) {
        const float sc = __ldg((x.kind == 1 ? p.k_scale : p.v_scale) + x.head);
        uint8_t* row = static_cast<uint8_t*>(pool) + at;
        *reinterpret_cast<uint2*>(row + ca) = quant8(xa, sc);
        *reinterpret_cast<uint2*>(row + cb) = quant8(xb, sc);
      } else {
        __nv_bfloat16* row = static_cast<__nv_bfloat16*>(pool) + at;
        *reinterpret_cast<uint4*>(row + ca) = rot ? pack8(xa) : a[i];
        *reinterpret_cast<uint4*>(row + cb) = rot ? pack8(xb) : b[i];
      }
    }
  }
}

// Any even rotary_dim, head_dim, alignment: one thread per pair of a head (or per
// two values past the rotated ones; one at an odd end).
template <bool INTERLEAVED, bool FP8>
__global__ void __launch_bounds__(kRopeThreads)
    rope_scalar_kernel(const __grid_constant__ RopeParams p) {
  const int64_t total = p.n_tokens * p.token_units;
  const int pairs = p.rotary / 2;
  for (int64_t i = blockIdx.x * (int64_t)kRopeThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kRopeThreads) {
    const int64_t t0 = i / p.token_units;
    const Unit x = locate(p, t0, (int)(i - t0 * p.token_units));
    const __nv_bfloat16* row =
        (x.kind == 0   ? p.q + x.token * p.q_stride
         : x.kind == 1 ? p.k + x.token * p.k_stride
                       : p.v + x.token * p.v_stride) + (int64_t)x.head * p.head_dim;
    const bool rot = x.kind != 2 && x.u < pairs;
    const int ca = !INTERLEAVED && rot ? x.u : 2 * x.u;
    const int cb = !INTERLEAVED && rot ? x.u + pairs : 2 * x.u + 1;
    const bool has_b = cb < p.head_dim;
    __nv_bfloat16 b0 = row[ca], b1 = has_b ? row[cb] : __nv_bfloat16();
    float y0 = __bfloat162float(b0), y1 = has_b ? __bfloat162float(b1) : 0.f;
    if (rot) {
      const float2 c = cos_sin(p.turns[x.u], __ldg(p.positions + x.token), p.amp, p.sign);
      const float x0 = y0, x1 = y1;
      y0 = x0 * c.x - x1 * c.y;
      y1 = x1 * c.x + x0 * c.y;
      b0 = __float2bfloat16_rn(y0);  // what is not turned keeps its bits
      b1 = __float2bfloat16_rn(y1);
    }
    if (x.kind == 0) {
      __nv_bfloat16* o = p.q_out + x.token * p.q_out_stride + (int64_t)x.head * p.head_dim;
      o[ca] = b0;
      if (has_b) o[cb] = b1;
      continue;
    }
    const int32_t slot = __ldg(p.slots + x.token);
    if (slot < 0 || slot >= p.num_slots) {
      if (x.head == 0 && x.u == 0) atomicOr(&g_rope_error, 1);
      continue;
    }
    const int64_t at = ((int64_t)slot * p.kv_heads + x.head) * p.head_dim;
    void* pool = x.kind == 1 ? p.k_pool : p.v_pool;
    if (FP8) {
      const float sc = __ldg((x.kind == 1 ? p.k_scale : p.v_scale) + x.head);
      unsigned short code;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(y1 / sc), "f"(y0 / sc));
      uint8_t* o = static_cast<uint8_t*>(pool) + at;
      o[ca] = (uint8_t)(code & 0xff);
      if (has_b) o[cb] = (uint8_t)(code >> 8);
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(pool) + at;
      o[ca] = b0;
      if (has_b) o[cb] = b1;
    }
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool INTERLEAVED, bool FP8>
int launch(RopeParams& p, bool vectors, cudaStream_t st) {
  const int heads = p.q_heads + 2 * p.kv_heads;
  if (!vectors) {
    p.head_units = (p.head_dim + 1) / 2;
    p.token_units = heads * p.head_units;
    const int64_t want = (p.n_tokens * p.token_units + kRopeThreads - 1) / kRopeThreads;
    const int blocks = (int)std::min<int64_t>(want, 16 * kSmCount);
    rope_scalar_kernel<INTERLEAVED, FP8><<<blocks, kRopeThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
  }
  p.head_units = p.head_dim / kUnit;
  p.token_units = heads * p.head_units;
  const int64_t total = p.n_tokens * p.token_units;
  // two units in flight per thread once the grid fills the SMs, else one (lower latency)
  const int ni = total >= (int64_t)kSmCount * 4 * kRopeThreads * 2 ? 2 : 1;
  p.cta_units = kRopeThreads * ni;
  p.cta_tokens = (p.cta_units - 1) / p.token_units + 2;
  // at most 34 KB: a token has at least rotary / 16 units
  const size_t smem = (size_t)p.cta_tokens * (p.rotary / 2) * sizeof(float2);
  const int64_t blocks = (total + p.cta_units - 1) / p.cta_units;
  if (blocks > INT32_MAX) return SEG_ATTN_ERR_UNSUPPORTED;
  if (ni == 2)
    rope_kernel<INTERLEAVED, FP8, 2><<<(unsigned)blocks, kRopeThreads, smem, st>>>(p);
  else
    rope_kernel<INTERLEAVED, FP8, 1><<<(unsigned)blocks, kRopeThreads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
}

int run(RopeParams& p, const seg_attn_rope_desc* rope, bool fp8, bool backward, void* stream) {
  if (!rope || rope->magic != SEG_ATTN_ROPE_MAGIC || rope->rotary_dim < 2 ||
      rope->rotary_dim > 2 * SEG_ATTN_ROPE_MAX_PAIRS || rope->rotary_dim % 2 != 0 ||
      (rope->layout != SEG_ATTN_ROPE_HALF && rope->layout != SEG_ATTN_ROPE_INTERLEAVED))
    return SEG_ATTN_ERR_INVALID_ARG;
  if (p.n_tokens < 0 || p.q_heads < 0 || p.kv_heads < 0 || p.head_dim < rope->rotary_dim ||
      p.num_slots < 0)
    return SEG_ATTN_ERR_INVALID_ARG;
  // the flat order of a token's units is counted in 32 bits
  if (p.head_dim > 4096 || p.q_heads > 65536 || p.kv_heads > 65536) return SEG_ATTN_ERR_UNSUPPORTED;
  const int64_t qw = (int64_t)p.q_heads * p.head_dim, kw = (int64_t)p.kv_heads * p.head_dim;
  if (p.n_tokens > 1 && ((p.q_heads > 0 && (p.q_stride < qw || p.q_out_stride < qw)) ||
                         (p.kv_heads > 0 && (p.k_stride < kw || p.v_stride < kw))))
    return SEG_ATTN_ERR_INVALID_ARG;
  if (p.n_tokens == 0 || p.q_heads + p.kv_heads == 0) return SEG_ATTN_OK;
  if (p.n_tokens > INT32_MAX) return SEG_ATTN_ERR_UNSUPPORTED;
  auto some = [](const void* x, uintptr_t a) { return x && aligned(x, a); };
  if (!some(p.positions, 4)) return SEG_ATTN_ERR_INVALID_ARG;
  if (p.q_heads > 0 && (!some(p.q, 2) || !some(p.q_out, 2))) return SEG_ATTN_ERR_INVALID_ARG;
  if (p.kv_heads > 0 && (!some(p.k, 2) || !some(p.v, 2) || !some(p.slots, 4) ||
                         !some(p.k_pool, fp8 ? 1 : 2) || !some(p.v_pool, fp8 ? 1 : 2) ||
                         (fp8 && (!some(p.k_scale, 4) || !some(p.v_scale, 4)))))
    return SEG_ATTN_ERR_INVALID_ARG;
  p.rotary = rope->rotary_dim;
  p.amp = rope->amp;
  p.sign = backward ? -1.f : 1.f;
  std::copy(rope->turns, rope->turns + p.rotary / 2, p.turns);
  auto rows = [&](const void* x, int64_t stride) {
    return aligned(x, 16) && (p.n_tokens == 1 || stride % 8 == 0);
  };
  bool vectors = p.head_dim % kUnit == 0 && p.rotary % kUnit == 0;
  if (p.q_heads > 0) vectors &= rows(p.q, p.q_stride) && rows(p.q_out, p.q_out_stride);
  if (p.kv_heads > 0)
    vectors &= rows(p.k, p.k_stride) && rows(p.v, p.v_stride) &&
               aligned(p.k_pool, fp8 ? 8 : 16) && aligned(p.v_pool, fp8 ? 8 : 16);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = rope->layout == SEG_ATTN_ROPE_INTERLEAVED;
  if (fp8) return inter ? launch<true, true>(p, vectors, st) : launch<false, true>(p, vectors, st);
  return inter ? launch<true, false>(p, vectors, st) : launch<false, false>(p, vectors, st);
}

RopeParams append_params(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                         const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                         const int32_t* positions, const int32_t* slots, int64_t n_tokens,
                         int q_heads, int kv_heads, int head_dim, void* k_pool, void* v_pool,
                         int64_t num_slots) {
  RopeParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_new);
  p.v = static_cast<const __nv_bfloat16*>(v_new);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slots;
  p.n_tokens = n_tokens;
  p.num_slots = num_slots;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.head_dim = head_dim;
  return p;
}

}  // namespace

int take_rope_error(int* value) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(int)) != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(int)) != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  *value = v;
  return SEG_ATTN_OK;
}

}  // namespace segattn

extern "C" int seg_attn_rope(const void* x, int64_t x_stride, void* out, int64_t out_stride,
                             const int32_t* positions, int64_t n_tokens, int heads, int head_dim,
                             const seg_attn_rope_desc* rope, int backward, void* stream) {
  if (backward != 0 && backward != 1) return SEG_ATTN_ERR_INVALID_ARG;
  if (heads <= 0) return SEG_ATTN_ERR_INVALID_ARG;
  segattn::RopeParams p =
      segattn::append_params(x, x_stride, out, out_stride, nullptr, 0, nullptr, 0, positions,
                             nullptr, n_tokens, heads, 0, head_dim, nullptr, nullptr, 0);
  return segattn::run(p, rope, false, backward != 0, stream);
}

extern "C" int seg_attn_rope_append(const void* q, int64_t q_stride, void* q_out,
                                    int64_t q_out_stride, const void* k_new, int64_t k_stride,
                                    const void* v_new, int64_t v_stride, const int32_t* positions,
                                    const int32_t* slots, int64_t n_tokens, int q_heads,
                                    int kv_heads, int head_dim, const seg_attn_rope_desc* rope,
                                    void* k_pool, void* v_pool, int64_t num_slots, void* stream) {
  if (kv_heads <= 0) return SEG_ATTN_ERR_INVALID_ARG;
  segattn::RopeParams p = segattn::append_params(
      q, q_stride, q_out, q_out_stride, k_new, k_stride, v_new, v_stride, positions, slots,
      n_tokens, q_heads, kv_heads, head_dim, k_pool, v_pool, num_slots);
  return segattn::run(p, rope, false, false, stream);
}

extern "C" int seg_attn_rope_append_fp8(
    const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k_new,
    int64_t k_stride, const void* v_new, int64_t v_stride, const int32_t* positions,
    const int32_t* slots, int64_t n_tokens, int q_heads, int kv_heads, int head_dim,
    const seg_attn_rope_desc* rope, const float* k_scale, const float* v_scale, void* k_pool,
    void* v_pool, int64_t num_slots, void* stream) {
  if (kv_heads <= 0) return SEG_ATTN_ERR_INVALID_ARG;
  segattn::RopeParams p = segattn::append_params(
      q, q_stride, q_out, q_out_stride, k_new, k_stride, v_new, v_stride, positions, slots,
      n_tokens, q_heads, kv_heads, head_dim, k_pool, v_pool, num_slots);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  return segattn::run(p, rope, true, false, stream);
}
