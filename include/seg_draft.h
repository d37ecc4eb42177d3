/*
 * seg_draft.h -- rotary positions and drafted tokens over the segmentable KV
 * cache (C ABI of libsegattn.so, beside seg_attn.h whose conventions hold:
 * the caller owns every buffer, nothing is allocated or synchronised, errors
 * are returned before anything is launched, device code never traps).
 *
 * One step of a serving loop that checks several drafted tokens per request
 * at once (lookahead decoding, Flood README feature list) uses them in turn:
 *   seg_attn_rope_append   rotate the new queries, write the rotated keys and
 *                          the values of the drafted tokens into their slots
 *   seg_attn_tree          attention of every drafted token over the cached
 *                          keys and its own ancestors among the drafts
 *   seg_attn_kv_move       move the accepted tokens' rows from the draft slots
 *                          to the end of the request's own run
 * Every call can be captured into a CUDA graph.
 */
#ifndef SEG_DRAFT_H_
#define SEG_DRAFT_H_

#include "seg_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Rotary positions.
 *
 * A head's first rotary_dim values are rotary_dim / 2 pairs; pair i of a token
 * at position p is turned by the angle p * w_i:
 *   y0 = amp * (x0 cos(p w_i) - x1 sin(p w_i))
 *   y1 = amp * (x1 cos(p w_i) + x0 sin(p w_i))
 * The values past rotary_dim are copied.  Layouts:
 *   SEG_ATTN_ROPE_HALF         pair i is (x[i], x[i + rotary_dim / 2])
 *   SEG_ATTN_ROPE_INTERLEAVED  pair i is (x[2 i], x[2 i + 1])
 * w_i = base^(-2 i / rotary_dim), changed by the scaling below.
 *
 * The plan keeps each w_i as the fraction of a turn per position, in units of
 * 2^-64: position times that, modulo 2^64, is the angle without any loss at
 * any int32 position (rounding of w_i itself: 2^-65 turns per position), and
 * needs no table of cosines in device memory.
 * ---------------------------------------------------------------------- */
enum { SEG_ATTN_ROPE_HALF = 0, SEG_ATTN_ROPE_INTERLEAVED = 1 };

/* Scalings for contexts longer than the original one.  f = factor, L =
 * original_len, T_i = L w_i / (2 pi) the turns pair i makes over L.
 *   NONE
 *   LINEAR      w_i / f (position interpolation)
 *   NTK         base * f^(rotary_dim / (rotary_dim - 2)) in place of base
 *   YARN        w_i (1 - r_i) + w_i / f r_i, where r_i rises linearly in i from
 *               0 at floor(pair(high)) to 1 at ceil(pair(low)), pair(t) =
 *               rotary_dim ln(L / (2 pi t)) / (2 ln base), both ends clamped to
 *               [0, rotary_dim - 1]; amp = 0.1 ln f + 1.  low / high: turns
 *               (0: 1 and 32)
 *   WAVELENGTH  w_i k_i + w_i / f (1 - k_i), k_i = (T_i - low) / (high - low)
 *               clamped to [0, 1].  low / high: turns (0: 1 and 4)
 *   PER_PAIR    w_i / factors[i]
 */
enum {
  SEG_ATTN_ROPE_SCALE_NONE = 0,
  SEG_ATTN_ROPE_SCALE_LINEAR = 1,
  SEG_ATTN_ROPE_SCALE_NTK = 2,
  SEG_ATTN_ROPE_SCALE_YARN = 3,
  SEG_ATTN_ROPE_SCALE_WAVELENGTH = 4,
  SEG_ATTN_ROPE_SCALE_PER_PAIR = 5
};

typedef struct seg_attn_rope_scaling {
  int32_t kind;          /* SEG_ATTN_ROPE_SCALE_* */
  int32_t num_factors;   /* PER_PAIR: rotary_dim / 2 */
  double factor;         /* f > 0 */
  double original_len;   /* L > 0 (YARN, WAVELENGTH) */
  double low, high;      /* low < high */
  double amp;            /* 0: the scaling's own (YARN as above, otherwise 1) */
  const double* factors; /* PER_PAIR: [num_factors], each > 0 (host) */
} seg_attn_rope_scaling;

#define SEG_ATTN_ROPE_MAGIC 0x45504f52u /* "ROPE" */
#define SEG_ATTN_ROPE_MAX_PAIRS 128

/* Filled by seg_attn_rope_plan; passed back unchanged.  A plain value: host
 * memory only, may be copied, nothing to free. */
typedef struct seg_attn_rope_desc {
  uint32_t magic;
  int32_t rotary_dim;    /* even, 2 .. 256 */
  int32_t layout;
  float amp;
  uint64_t turns[SEG_ATTN_ROPE_MAX_PAIRS]; /* 2^-64 turns per position */
} seg_attn_rope_desc;

/* Host only.  base > 1 and finite; scaling NULL = NONE.  An odd or
 * out-of-range rotary_dim returns SEG_ATTN_ERR_UNSUPPORTED. */
int seg_attn_rope_plan(int rotary_dim, int layout, double base,
                       const seg_attn_rope_scaling* scaling, seg_attn_rope_desc* desc);

/*
 * seg_attn_rope -- rotate bf16 rows.
 *   x, out       bf16, `heads` heads of head_dim consecutive values per token;
 *                token t starts at t * x_stride (out_stride) elements, so x may
 *                be the query part of a fused projection.  out may be x with the
 *                same stride (in place; another stride is refused); otherwise
 *                they must not overlap.
 *   positions    int32 [n_tokens] (device); any value, negative ones included
 *   backward     0: the rotation above; 1: its transpose (the gradient of x
 *                given the gradient of out)
 * head_dim >= rotary_dim; strides >= heads * head_dim (ignored for one token).
 * Products in fp32, one rounding to bf16.  Rows whose addresses, strides,
 * head_dim and rotary_dim are multiples of 16 bytes / 16 elements move as
 * 16-byte vectors; others take a slower element-wise kernel.
 */
int seg_attn_rope(const void* x, int64_t x_stride, void* out, int64_t out_stride,
                  const int32_t* positions, int64_t n_tokens, int heads, int head_dim,
                  const seg_attn_rope_desc* rope, int backward, void* stream);

/*
 * seg_attn_rope_append -- seg_attn_kv_append with the rotation on the way, in
 * one launch: q_out = rotated q; k_pool[slots[t]] = rotated k_new; v_pool[
 * slots[t]] = v_new.  Strides as in seg_attn_rope (the three inputs may be the
 * parts of one fused projection); the pools are dense as in seg_attn.h.
 * q_heads may be 0 (q and q_out unused).  q_out may be q with the same stride.
 * A slot outside [0, num_slots) writes no cache row (its q_out row is written)
 * and sets value 2 of the device error word.  A slot listed twice ends with
 * values of either token.
 */
int seg_attn_rope_append(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                         const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                         const int32_t* positions, const int32_t* slots, int64_t n_tokens,
                         int q_heads, int kv_heads, int head_dim, const seg_attn_rope_desc* rope,
                         void* k_pool, void* v_pool, int64_t num_slots, void* stream);

/*
 * seg_attn_rope_append_fp8 -- the same into E4M3 pools: code =
 * round-to-nearest-even(value / scale[head]) saturated to +-448, with the
 * rotated key rounded once, from fp32 (seg_attn_kv_append_fp8's codes for an
 * unrotated value).  Scales are device values, finite and > 0 (a head of zeros
 * takes any positive one); they are not checked.
 */
int seg_attn_rope_append_fp8(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                             const void* k_new, int64_t k_stride, const void* v_new,
                             int64_t v_stride, const int32_t* positions, const int32_t* slots,
                             int64_t n_tokens, int q_heads, int kv_heads, int head_dim,
                             const seg_attn_rope_desc* rope, const float* k_scale,
                             const float* v_scale, void* k_pool, void* v_pool, int64_t num_slots,
                             void* stream);

/* ------------------------------------------------------------------------
 * Attention of drafted tokens.
 *
 * Request r has draft_lens[r] drafted tokens; their K/V rows are the last
 * draft_lens[r] logical keys of its segment list, after P_r cached keys.
 * Drafted token i sees every cached key and the drafted keys of its mask:
 *   parents     parent of each drafted token, -1 (the last cached token) or a
 *               smaller index of the same request: i sees itself and its
 *               ancestors
 *   mask        [sum draft_lens[r]^2] bytes, per request row-major: i sees j
 *               where the byte is not 0 (a token need not see itself)
 *   neither     a chain: i sees 0 .. i
 * Scores, their maximum and sum and the output are accumulated in fp32.  A
 * softmax weight is rounded to the 16-bit operand of its product with V: bf16
 * over a bf16 cache (2^-8 of the weight), f16 over an E4M3 cache (2^-11; queries
 * are f16 there too, so |q| must be below 65504).  The sum divides by the
 * unrounded weights, and out rounds to bf16 once.
 * out and lse as in seg_attn.h; a token that sees no key (P_r = 0 and an empty
 * mask row) gets out = 0 and lse = -inf.  What a token does not see, NaN and
 * infinities included, never reaches its row.
 * ---------------------------------------------------------------------- */
#define SEG_ATTN_TREE_MAGIC 0x54524545u /* "TREE" */
#define SEG_ATTN_TREE_VERSION 1u
#define SEG_ATTN_TREE_MAX_DRAFT 1024

typedef struct seg_attn_tree_desc {
  uint32_t magic, version;
  int32_t batch, max_draft;
  int64_t off_mask;       /* mask rows, requests back to back: ceil(draft_len / 32) words
                             each, bit j of word w of row i: i sees drafted token 32 w + j */
  int64_t off_draft_slot; /* [total_q] pool slot of each drafted token */
  seg_attn_table_desc pass; /* the prefill table of all keys (offsets into the same buffer;
                               for the tree calls only: the plain ones refuse it);
                               words 13, 14 of a work row: first mask word of the request
                               (low and high half) */
  uint64_t table_bytes, workspace_bytes;
} seg_attn_tree_desc;

/*
 * seg_attn_build_tree_table -- host only; arguments, errors and use of host_out
 * as seg_attn_build_table.  draft_lens[r] in 0 .. SEG_ATTN_TREE_MAX_DRAFT and at most the
 * request's keys (SEG_ATTN_ERR_QLEN_GT_KLEN otherwise); at most one of parents
 * and mask.  Shapes: head_dim 64 or 128, q_heads / kv_heads a power of two <= 128.
 */
int seg_attn_build_tree_table(int batch, const int32_t* draft_lens, const int32_t* parents,
                              const uint8_t* mask, const int32_t* seg_counts,
                              const int32_t* seg_starts, const int32_t* seg_lens,
                              int64_t num_slots, int q_heads, int kv_heads, int head_dim,
                              void* host_out, size_t host_out_bytes, seg_attn_tree_desc* desc);

/* Device workspace (bytes) the tree calls need; 0 if none. */
size_t seg_attn_tree_workspace_size(const seg_attn_tree_desc* desc);

/*
 * seg_attn_tree / seg_attn_tree_fp8 -- arguments as seg_attn_prefill /
 * seg_attn_prefill_fp8, with a tree table.  Two calls that may overlap on the
 * GPU need workspaces of their own.  Scales as in seg_attn_rope_append_fp8.
 */
int seg_attn_tree(const void* q, const void* k_pool, const void* v_pool, void* out, float* lse,
                  const void* dev_table, const seg_attn_tree_desc* desc, float softmax_scale,
                  void* workspace, size_t workspace_bytes, void* stream);
int seg_attn_tree_fp8(const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
                      const float* v_scale, void* out, float* lse, const void* dev_table,
                      const seg_attn_tree_desc* desc, float softmax_scale, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * seg_attn_kv_move -- copy cache rows from slot to slot: k_pool[dst[i]] =
 * k_pool[src[i]], v_pool likewise.
 *   src, dst     int32 [n_moves] (device).  src == dst (-1 included) moves
 *                nothing; otherwise a slot outside [0, num_slots) skips the move
 *                and sets value 2 of the device error word.
 *   offsets      int32 [n_groups + 1] (device), non-decreasing from 0: moves
 *                offsets[g] .. offsets[g + 1] - 1 are done in that order, as long
 *                as no move reads a row that an earlier move of its group wrote
 *                (moving accepted rows towards the front never does); values
 *                outside [0, n_moves] are clamped.  NULL: every move is a
 *                group of its own (n_groups is ignored).
 *                Groups run in any order: no group may touch a row that
 *                another one writes.
 *   elem_bytes   2 (bf16 pools) or 1 (E4M3); kv_heads * head_dim * elem_bytes
 *                must be a multiple of 16
 */
int seg_attn_kv_move(void* k_pool, void* v_pool, const int32_t* src, const int32_t* dst,
                     int64_t n_moves, const int32_t* offsets, int64_t n_groups, int kv_heads,
                     int head_dim, int elem_bytes, int64_t num_slots, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SEG_DRAFT_H_ */
