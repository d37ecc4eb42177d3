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

// 128 threads with two units each: 83.8 us for 16381 tokens x 64 heads (6.4 TB/s, 0.98 of
// the copy rate), one unit 93.1.  Measured beside an earlier form of 88.8 us: 256 threads
// 91.5, 64 threads 90.8, four units 95.0; warps that own a token without a barrier 97, a
// persistent grid with the next loads in flight 94.
constexpr int kRopeThreads = 128;
constexpr int kScalarThreads = 256;
constexpr int kUnit = 16;  // values per unit

// Division of x < 2^31 by a launch constant d: m = floor(2^(32 + s) / d) + 1 with
// 2^s < d <= 2^(s + 1) exceeds 2^(32 + s) / d by e / d, e <= d, and x e < 2^(32 + s), so
// the product's upper bits are the quotient (Granlund and Montgomery's method).
struct FastDiv {
  uint32_t m;  // 0: d = 1
  uint32_t s;
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
    return m ? __umulhi(x, m) >> s : x;
  }
};
FastDiv fast_div(uint32_t d) {
  FastDiv f = {0, 0};
  if (d == 1) return f;
  while ((2ull << f.s) < d) ++f.s;
  f.m = (uint32_t)((1ull << (32 + f.s)) / d + 1);
  return f;
}

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
  FastDiv by_head, by_token;       // divisions by them
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

// Packed fp32 pairs: one instruction does two products or fused products.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// x / scale, rounded as the division is: a product with the rounded reciprocal, then one
// correction by the remainder (Markstein's theorem: correctly rounded when the
// reciprocal is).  The remainder is taken with the product's sign (q scale - x), so that a
// zero one adds -0 and a product of -0 stays -0, whose code is 0x80.  An infinite or NaN
// product has no remainder and is kept.
__device__ __forceinline__ float quotient(float x, float scale, float reciprocal) {
  const float q = x * reciprocal;
  const float r = fmaf(fmaf(q, scale, -x), -reciprocal, q);
  return fabsf(q) < 3.0e38f ? r : q;
}
// E4M3 codes of four values over the head's scale, as seg_attn_kv_append_fp8's.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float scale,
                                           float reciprocal) {
  float x[4] = {a, b, c, d};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    // outside this range the reciprocal, or the remainder, is not a normal number
    x[i] = scale > 1e-18f && scale < 1e18f ? quotient(x[i], scale, reciprocal) : x[i] / scale;
  unsigned short lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Where a unit of the flat order (token, then query heads, key heads, value
// heads, then units of the head) lives.
struct Unit {
  int64_t token;
  int head;   // of its kind
  int kind;   // 0 query, 1 key, 2 value
  int u;      // unit of the head
};
__device__ __forceinline__ Unit locate(const RopeParams& p, int64_t t0, uint32_t at) {
  Unit x;
  const uint32_t tl = p.by_token(at);
  const uint32_t rest = at - tl * p.token_units;
  const int h = (int)p.by_head(rest);
  x.u = (int)rest - h * p.head_units;
  x.token = t0 + tl;
  x.kind = h < p.q_heads ? 0 : h < p.q_heads + p.kv_heads ? 1 : 2;
  x.head = h - (x.kind == 0 ? 0 : x.kind == 1 ? p.q_heads : p.q_heads + p.kv_heads);
  return x;
}

// NI: units per thread.
template <bool INTERLEAVED, bool FP8, int NI>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  // [tokens of this CTA][8][rotary / 16]: pair 8 u + e of a token at e * (rotary / 16) + u,
  // so that the units u of neighbouring lanes read neighbouring values
  extern __shared__ float2 cs[];
  constexpr uint32_t kCtaUnits = kRopeThreads * NI;
  const uint32_t first = blockIdx.x * kCtaUnits;  // a launch has < 2^31 units
  const int count = (int)min(kCtaUnits, (uint32_t)p.n_tokens * p.token_units - first);
  const uint32_t t0 = p.by_token(first);
  const int off0 = (int)(first - t0 * p.token_units);
  const int pairs = p.rotary / 2, rot_units = p.rotary / kUnit;

  uint4 a[NI], b[NI];
  Unit un[NI];
  int32_t slot[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int at = i * kRopeThreads + threadIdx.x;
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
  const int tokens = (int)p.by_token(off0 + count - 1) + 1;
  for (int i = threadIdx.x; i < tokens * pairs; i += kRopeThreads) {
    const int t = i / pairs, j = i - t * pairs;
    cs[t * pairs + (j & 7) * rot_units + (j >> 3)] =
        cos_sin(p.turns[j], __ldg(p.positions + t0 + t), p.amp, p.sign);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const Unit& x = un[i];
    if (x.kind < 0) continue;
    const bool rot = x.kind != 2 && x.u < rot_units;
    const bool split = !INTERLEAVED && rot;
    const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
    const uint32_t wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
    // the unit's values: first sides f, second sides g of pairs (2 e, 2 e + 1)
    float2 f[4], g[4];
    const float2* c = cs + (int)(x.token - t0) * pairs + x.u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (INTERLEAVED) {
        const uint32_t w0 = e < 2 ? wa[2 * e] : wb[2 * e - 4];
        const uint32_t w1 = e < 2 ? wa[2 * e + 1] : wb[2 * e - 3];
        f[e] = make_float2(bf_lo(w0), bf_lo(w1));
        g[e] = make_float2(bf_hi(w0), bf_hi(w1));
      } else {
        f[e] = make_float2(bf_lo(wa[e]), bf_hi(wa[e]));
        g[e] = make_float2(bf_lo(wb[e]), bf_hi(wb[e]));
      }
      if (rot) {
        const float2 p0 = c[2 * e * rot_units], p1 = c[(2 * e + 1) * rot_units];
        const uint64_t cc = pack2(p0.x, p1.x);
        const uint64_t f2 = pack2(f[e].x, f[e].y), g2 = pack2(g[e].x, g[e].y);
        f[e] = unpack2(fma2(g2, pack2(-p0.y, -p1.y), mul2(f2, cc)));
        g[e] = unpack2(fma2(f2, pack2(p0.y, p1.y), mul2(g2, cc)));
      }
    }
    uint4 oa = a[i], ob = b[i];  // what is not turned keeps its bits
    if (rot && (x.kind == 0 || !FP8)) {
      if (INTERLEAVED) {
        oa = make_uint4(bf_pack(f[0].x, g[0].x), bf_pack(f[0].y, g[0].y),
                        bf_pack(f[1].x, g[1].x), bf_pack(f[1].y, g[1].y));
        ob = make_uint4(bf_pack(f[2].x, g[2].x), bf_pack(f[2].y, g[2].y),
                        bf_pack(f[3].x, g[3].x), bf_pack(f[3].y, g[3].y));
      } else {
        oa = make_uint4(bf_pack(f[0].x, f[0].y), bf_pack(f[1].x, f[1].y),
                        bf_pack(f[2].x, f[2].y), bf_pack(f[3].x, f[3].y));
        ob = make_uint4(bf_pack(g[0].x, g[0].y), bf_pack(g[1].x, g[1].y),
                        bf_pack(g[2].x, g[2].y), bf_pack(g[3].x, g[3].y));
      }
    }
    const int ca = split ? 8 * x.u : kUnit * x.u, cb = split ? ca + pairs : ca + 8;
    if (x.kind == 0) {
      __nv_bfloat16* row = p.q_out + x.token * p.q_out_stride + x.head * p.head_dim;
      *reinterpret_cast<uint4*>(row + ca) = oa;
      *reinterpret_cast<uint4*>(row + cb) = ob;
      continue;
    }
    if (slot[i] < 0 || slot[i] >= p.num_slots) {
      if (x.head == 0 && x.u == 0) atomicOr(&g_rope_error, 1);
      continue;
    }
    const int64_t at = ((int64_t)slot[i] * p.kv_heads + x.head) * p.head_dim;
    void* pool = x.kind == 1 ? p.k_pool : p.v_pool;
    if (FP8) {
      const float sc = __ldg((x.kind == 1 ? p.k_scale : p.v_scale) + x.head), rc = 1.f / sc;
      uint8_t* row = static_cast<uint8_t*>(pool) + at;
      uint2 qa, qb;
      if (INTERLEAVED) {
        qa = make_uint2(quant4(f[0].x, g[0].x, f[0].y, g[0].y, sc, rc),
                        quant4(f[1].x, g[1].x, f[1].y, g[1].y, sc, rc));
        qb = make_uint2(quant4(f[2].x, g[2].x, f[2].y, g[2].y, sc, rc),
                        quant4(f[3].x, g[3].x, f[3].y, g[3].y, sc, rc));
      } else {
        qa = make_uint2(quant4(f[0].x, f[0].y, f[1].x, f[1].y, sc, rc),
                        quant4(f[2].x, f[2].y, f[3].x, f[3].y, sc, rc));
        qb = make_uint2(quant4(g[0].x, g[0].y, g[1].x, g[1].y, sc, rc),
                        quant4(g[2].x, g[2].y, g[3].x, g[3].y, sc, rc));
      }
      *reinterpret_cast<uint2*>(row + ca) = qa;
      *reinterpret_cast<uint2*>(row + cb) = qb;
    } else {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(pool) + at;
      *reinterpret_cast<uint4*>(row + ca) = oa;
      *reinterpret_cast<uint4*>(row + cb) = ob;
    }
  }
}

// Any even rotary_dim, head_dim, alignment: one thread per pair of a head (or per
// two values past the rotated ones; one at an odd end).
template <bool INTERLEAVED, bool FP8>
__global__ void __launch_bounds__(kScalarThreads)
    rope_scalar_kernel(const __grid_constant__ RopeParams p) {
  const int64_t total = p.n_tokens * p.token_units;
  const int pairs = p.rotary / 2;
  for (int64_t i = blockIdx.x * (int64_t)kScalarThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kScalarThreads) {
    const int64_t t0 = i / p.token_units;
    const Unit x = locate(p, t0, (uint32_t)(i - t0 * p.token_units));
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
    p.by_head = fast_div(p.head_units);
    p.by_token = fast_div(p.token_units);
    const int64_t want = (p.n_tokens * p.token_units + kScalarThreads - 1) / kScalarThreads;
    const int blocks = (int)std::min<int64_t>(want, 16 * kSmCount);
    rope_scalar_kernel<INTERLEAVED, FP8><<<blocks, kScalarThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
  }
  p.head_units = p.head_dim / kUnit;
  p.token_units = heads * p.head_units;
  p.by_head = fast_div(p.head_units);
  p.by_token = fast_div(p.token_units);
  const int64_t all = p.n_tokens;
  // two units in flight per thread in long calls, one in short ones, where latency counts
  // (one unit against two, us: one token 2.6 / 3.1, 128 tokens of 64 + 8 + 8 heads 3.0 / 3.3,
  // 1024 of them 9.0 / 8.3, 16381 tokens of 64 heads 93.1 / 83.8)
  const int ni = all * p.token_units >= (int64_t)kSmCount * 8 * kRopeThreads * 2 ? 2 : 1;
  const int cta_units = kRopeThreads * ni;
  const int cta_tokens = (cta_units - 1) / p.token_units + 2;  // the most that a CTA touches
  // at most 18.2 KB: a token has at least rotary / 16 units
  const size_t smem = (size_t)cta_tokens * (p.rotary / 2) * sizeof(float2);
  // a launch counts its units in 31 bits: more tokens take several
  const int64_t most = (INT32_MAX - cta_units) / p.token_units;
  for (int64_t done = 0; done < all; done += p.n_tokens) {
    p.n_tokens = std::min(all - done, most);
    const unsigned blocks =
        (unsigned)((p.n_tokens * p.token_units + cta_units - 1) / cta_units);
    if (ni == 2)
      rope_kernel<INTERLEAVED, FP8, 2><<<blocks, kRopeThreads, smem, st>>>(p);
    else
      rope_kernel<INTERLEAVED, FP8, 1><<<blocks, kRopeThreads, smem, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SEG_ATTN_ERR_CUDA;
    if (p.q_heads > 0) {
      p.q += p.n_tokens * p.q_stride;
      p.q_out += p.n_tokens * p.q_out_stride;
    }
    if (p.kv_heads > 0) {
      p.k += p.n_tokens * p.k_stride;
      p.v += p.n_tokens * p.v_stride;
      p.slots += p.n_tokens;
    }
    p.positions += p.n_tokens;
  }
  return SEG_ATTN_OK;
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
  // in place with another stride, a token's output would lie over other tokens' input
  if (p.n_tokens > 1 && p.q_heads > 0 && p.q && p.q == p.q_out && p.q_stride != p.q_out_stride)
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
