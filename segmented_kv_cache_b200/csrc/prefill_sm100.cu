// Chunked-prefill SegmentAttention for sm_100a (tcgen05 + TMEM + TMA).
//
// Work item = (request, kv head g, two query tiles).  A query tile is 128
// rows of (query, head) pairs: 128/G consecutive queries x the G query heads
// that share kv head g, so every K/V byte fetched serves all G heads, and a
// small chunk (few new queries per request) still fills the 128 rows.  The
// two tiles share each K/V tile, which halves L2->SM traffic per flop.
//
// K/V tiles are 128 consecutive *logical* keys.  Segments (Flood README,
// "Introduction": contiguous runs in a shared slot pool) make every row's
// slot known up front.  A tile whose 128 keys are 128 consecutive pool slots
// (the common case: segments are long) is loaded as two tiled boxes straight
// into the 128-byte swizzled layout the tensor cores read; a tile that
// straddles segments as boxes of 32 and 8 keys where the slots allow it and
// TMA gather4 (four pool rows per instruction) where they do not.  Keys past
// the end of the request are clamped to its last key and masked.
//
// Warp roles (two query tiles: 10 warps, 12 over an FP8 cache; one: 6 and 8):
//   warp 0       TMA producer: Q tiles once, then a K ring and a V ring
//                (depths below), K tile i + 1 before V tile i.
//   warp 1       TMEM allocator and MMA issuer: the whole warp runs the issue
//                loop, one elected lane executes each tcgen05.mma / commit.
//   warps 2-5    softmax for query tile 0, warps 6-9 for tile 1: one thread
//                per row (its TMEM lane); online softmax (running max m and
//                normaliser l, as in the Ascend FlashAttention article,
//                "bottleneck 2") in registers, O rescaled in TMEM only when
//                the max grows by more than 2^8 (the final O / l uses the same
//                reference max, so the result is unchanged), epilogue O / l ->
//                bf16 and lse.
// Two query tiles (the usual item):
//                  S   = Q_t K^T   (SS: Q tile and K stage from shared memory)
//                  O_t += P_t V    (TS: P from tensor memory, V MN-major)
// and the two tiles take turns on one S buffer.  A softmax thread loads its
// whole S row, releases the buffer (the other tile's QK can go), and writes P
// into tensor-memory columns of its own, so the next K tile's S of a query
// tile is computed while this tile's softmax still runs, and no MMA writes
// tensor memory that an earlier MMA reads (such a write waits for the tensor
// pipe to drain).  P stays out of shared memory, whose bandwidth the SS QK,
// the V reads of PV and the TMA writes already share.
// TMEM columns: O0 [0,128) O1 [128,256) S [256,384) P0 [384,448) P1 [448,512).
// One query tile: S double-buffered, each buffer with a P region of its own, so
// the QK that refills an S buffer never overwrites what the PV before it reads.
// TMEM columns: O [0,128) P0 [128,192) P1 [192,256) S0 [256,384) S1 [384,512).
// Over an FP8 cache the last two warps widen the E4M3 codes of K and of V tiles to f16
// in place, inside the ring slot whose second half the codes were loaded into.  (A single
// staging tile per K and V, as the one-tile kernel had, exposed every tile's load latency:
// 64 trees of 16 over 4k keys, 308 us; now 206.)
// Drafted tokens (TREE, see the kernel's comment): masks of bits on the last K tiles, and
// items of one query tile run both softmax groups on it.
// Every mbarrier wait is bounded (1 s); a timeout stops all roles of the CTA,
// drains in-flight copies and MMAs, frees TMEM and flags a device error.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <type_traits>
#include <utility>

#include "ptx_sm100.cuh"
#include "seg_attn_internal.h"

namespace segattn {

__device__ int g_device_error;  // non-zero once a bounded wait gave up

namespace {

// Warps: producer, MMA issuer, four softmax warps per query tile, and over an FP8 cache
// one warp that widens the E4M3 codes of K tiles and one for V tiles.  Registers are dealt
// out per SM sub-partition: 6 or 8 warps leave the one-tile kernels 255 per thread (no
// spills), 9 to 12 warps 168.
template <bool SINGLE>
constexpr int conv_warp0() {
  return SINGLE ? 6 : 10;
}
template <bool SINGLE, bool FP8>
constexpr int cta_threads() {
  return (conv_warp0<SINGLE>() + (FP8 ? 2 : 0)) * 32;
}
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // default limit of a bounded wait
// Stall test (off by default): the K tile at which every later prefill CTA's
// producer stops loading (-1: none), and the limit of its bounded waits.
std::atomic<int> g_stall_tile{-1};
std::atomic<uint64_t> g_stall_wait_ns{kWaitLimitNs};
// Order test (off by default): every softmax warp of a one-tile item sleeps this
// long after it signals P of the item's last K tile.
std::atomic<int> g_order_delay_ns{0};
constexpr float kRescaleLog2 = 8.0f;
constexpr uint32_t kHalfBytes = 128 * 128;  // 128 rows x 64 bf16 (one swizzle-128B panel)

// Tensor maps of one pool: single rows (gathered four at a time) and boxes of 8, 32 and
// 128 consecutive slots of one kv head.
struct PoolMaps {
  CUtensorMap row, box8, box32, box128;
};

struct PrefillParams {
  __nv_bfloat16* out;
  float* lse;
  TableView tab;
  float scale_log2;
  int q_heads, kv_heads, group, qpt, causal;
  float* part_o;    // split items: [slot][kItemRows][D], O / l of the piece
  float* part_lse;  // split items: [slot][kItemRows], log2 of the piece's sum of exp
  int work_base;    // first work item of this launch
  const float* k_scale;  // FP8 cache: [kv_heads] dequantisation scales (value = code * scale)
  const float* v_scale;
  uint64_t wait_ns;      // limit of every bounded wait (1 s unless a stall test shortens it)
  int withhold_tile;     // stall test: the producer stops before loading this K tile (-1: off)
  int p_delay_ns;        // order test: one-tile softmax sleep after the last P is signalled (0: off)
  const uint32_t* mask_base;   // drafted tokens: the table, whose words hold the mask rows
  const int32_t* draft_slot;   // drafted tokens: [total_q] pool slot of each
  const void* v_pool;          // drafted tokens: V rows by address (the rare path of add_nonfinite)
};

// Query region (one Q tile or two) + K ring + V ring + barriers + alignment slack.
// The d = 64 variant asks for more than half the SM's shared memory as well, so one
// CTA owns an SM and its 512 tensor-memory columns.
// K/V ring depths (stages of K, of V).  The one-tile kernel spends the second query
// tile's space on a third V stage; the two-tile kernels' QK of a K tile runs a softmax
// ahead of the PV of the previous one, so K tiles are wanted earlier than V tiles.
constexpr int kRingK = 3;
template <bool SINGLE>
constexpr int ring_v() {
  return SINGLE ? 3 : 2;
}

// An FP8 cache's E4M3 codes of a K/V tile land in the second half of its ring slot and
// are widened to f16 there, so as many tiles are in flight as over a bf16 cache.
constexpr size_t kBarrierBytes = 512;  // mbarriers, tensor-memory address, flags

template <int D, bool SINGLE>
constexpr size_t query_region_bytes() {
  return (SINGLE ? 1 : 2) * (D / 64) * (size_t)kHalfBytes;
}

template <int D, bool SINGLE>
constexpr size_t prefill_smem_bytes() {
  constexpr size_t need = query_region_bytes<D, SINGLE>() +
                          (kRingK + ring_v<SINGLE>()) * (D / 64) * (size_t)kHalfBytes +
                          kBarrierBytes + 1024;
  static_assert(need <= 227 * 1024, "shared memory per CTA");
  return need < 120 * 1024 ? 120 * 1024 : need;
}

// Three-input maximum (one instruction on sm_100).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Packed fp32 pairs: one instruction does two fmaf / two adds, each rounded as
// the scalar one would be.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Eight bf16 (one 16-byte chunk) -> eight f16 in place; exact for |x| in
// [2^-14, 65504], rounded below (f16 subnormals), infinite above.
__device__ __forceinline__ void bf16x8_to_f16x8(uint4& v) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = ptx::pack_f16x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// The E4M3 codes of one tile, in the second half of a ring slot (kTileKeys rows of D
// bytes, plain row-major) -> f16 over the whole slot in the 128-byte-swizzled K-major
// layout the tensor cores read (the layout a tiled TMA load of a bf16 tile produces):
// row r, 16-byte chunk c of 64-column half h lands at h * kHalfBytes + r * 128 +
// ((c ^ (r & 7)) * 16).  One warp walks the tile in passes of 8 rows; a lane has one
// 16-code column j of row r0 (and, d = 128, r0 + 4), so its offsets are those of the
// first pass plus a constant.  In place needs no barrier across warps: with d = 128 a
// row's codes lie exactly under its own second half; with d = 64 the output of row r
// covers the codes of rows 2 r - 128 and 2 r - 127, never later than r; so it is enough
// that the warp has loaded a pass before it stores that pass.  The eight lanes of a row
// (d = 128) hold columns of both halves, whose chunks share banks: the second half's
// lanes take the neighbouring row (r0 ^ 1), which turns their even chunks into odd ones,
// so loads and stores are both free of conflicts.
// One warp per K and per V tile instead of 64 threads per tile with two barriers: the
// chain of waits, barriers and latencies (1200 cycles a tile, K and V in turn) bounded
// both kernels.
template <int D>
__device__ __forceinline__ void widen_tile(uint8_t* slot, int lane) {
  constexpr int kCols = D / 16;             // 16-code columns of a row
  constexpr int kRowStep = 32 / kCols;      // rows of one load: 4 (d = 128) or 8 (d = 64)
  constexpr int kBatch = 32 / kRowStep;     // loads in flight per thread: 32 rows
  const int j = lane % kCols, r0 = (lane / kCols) ^ (j >> 2);
  const int c0 = (j & 3) * 2;
  const uint8_t* s = slot + (D / 64) * kHalfBytes / 2 + r0 * D + 16 * j;
  uint8_t* d = slot + (j >> 2) * kHalfBytes + r0 * 128;
#pragma unroll 1
  for (int r = 0; r < kTileKeys; r += 32, s += 32 * D, d += 32 * 128) {
    uint4 w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      w[k] = *reinterpret_cast<const uint4*>(s + k * kRowStep * D);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int sw = (r0 + k * kRowStep) & 7;
      uint4 lo, hi;
      ptx::e4m3x4_to_f16x4(w[k].x, lo.x, lo.y);
      ptx::e4m3x4_to_f16x4(w[k].y, lo.z, lo.w);
      ptx::e4m3x4_to_f16x4(w[k].z, hi.x, hi.y);
      ptx::e4m3x4_to_f16x4(w[k].w, hi.z, hi.w);
      *reinterpret_cast<uint4*>(d + k * kRowStep * 128 + ((c0 ^ sw) << 4)) = lo;
      *reinterpret_cast<uint4*>(d + k * kRowStep * 128 + (((c0 + 1) ^ sw) << 4)) = hi;
    }
  }
}

// SINGLE: every item of the launch has queries in its first query tile only
// (the planner lists those items last and launches them separately, so each
// instantiation keeps its own register allocation).
// FP8: the pools hold E4M3 codes (value = code * scale of the kv head).  Code
// tiles are loaded by TMA as raw bytes and widened to f16 (exact) in the K/V ring
// slots by the last warps; queries are converted bf16 -> f16 in shared memory
// and P is f16, so every product is f16 x f16 -> f32.  The K scale is folded
// into the softmax scale, the V scale into the output.
// TREE: the last q_len keys of a request are its drafted tokens, the queries of this
// call; a query sees every key before them and those its mask row has bits for.  Only
// the K tiles that reach past the cached keys look at the mask.  P of a masked key is
// an exact zero, but zero times an infinite or NaN value would still reach the row in
// P.V, so in those tiles non-finite values of drafted keys are replaced by zeros in the
// V tile, and the rows that do see such a key get them added at the end.
template <int D, bool SINGLE, bool FP8, bool TMA_OUT, bool TREE>
__global__ void __launch_bounds__(cta_threads<SINGLE, FP8>(), 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ PoolMaps tm_k, const __grid_constant__ PoolMaps tm_v,
                   const PrefillParams p) {
  using namespace ptx;
  constexpr int HALVES = D / 64;
  constexpr uint32_t TILE = HALVES * kHalfBytes;
  constexpr int KSTEPS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  constexpr int RK = kRingK, RV = ring_v<SINGLE>();
  constexpr int kConvWarp0 = conv_warp0<SINGLE>();
  // Q tiles at sQ + t * TILE.  Two query tiles (QT): P_t in tensor memory columns
  // [384 + 64 t, 448 + 64 t).
  constexpr bool QT = !SINGLE;
  constexpr uint32_t QSTRIDE = TILE;
  uint8_t* sQ = sm;
  uint8_t* sK = sm + query_region_bytes<D, SINGLE>();
  uint8_t* sV = sK + RK * TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + RV * TILE);
  uint64_t* q_full = bars + 0;
  uint64_t* k_full = bars + 1;    // [RK]
  uint64_t* k_empty = bars + 4;   // [RK]
  uint64_t* v_full = bars + 7;    // [RV]
  uint64_t* v_empty = bars + 10;  // [RV]
  uint64_t* s_full = bars + 13;   // [2] per query tile (S buffer)
  uint64_t* p_full = bars + 15;   // [2]
  uint64_t* o_full = bars + 17;   // [2]
  uint64_t* mma_done = bars + 19;
  uint64_t* code_k = bars + 20;     // FP8: [RK] codes landed in a K ring slot
  uint64_t* code_v = bars + 30;     // FP8: [RV] the same for V
  uint64_t* q_conv = bars + 24;     // FP8: queries converted to f16 in place
  uint64_t* s_free = bars + 25;     // two tiles: the shared S buffer read by its softmax
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 28);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* nonfinite = reinterpret_cast<int*>(bars + 34);  // TREE: some drafted V value was not finite
  volatile uint64_t* mask_at = bars + 36;  // TREE: first mask word of the request
  // limit of every bounded wait, read only when a wait checks it
  volatile uint64_t* wait_limit = reinterpret_cast<volatile uint64_t*>(bars + 29);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // drafted tokens: launched as a programmatic dependent, so that the launch itself
  // overlaps the end of whatever ran before; nothing is read or written before this
  if (TREE) grid_dependency_wait();
  // piece: keys tiles [kt0, kt1) of item (request, kv head g, query tiles from q0);
  // slot >= 0 when the item is split and this piece writes a partial result.  The
  // row also carries the request's first query row, queries, keys and the segment
  // of the piece's first key, so no dependent table load precedes the first copies.
  const int item = p.work_base + blockIdx.x;
  const int4 w0 = p.tab.work[4 * item], w1 = p.tab.work[4 * item + 1];
  const int4 w2 = p.tab.work[4 * item + 2], w3 = p.tab.work[4 * item + 3];
  const int g = w0.y, q0 = w0.z, kt0 = w0.w, slot = w1.y;
  const int n_tiles = w1.x - kt0;
  const int tok0 = w2.x, q_len = w2.y, k_len = w2.z;
  // Only query tile 0 holds queries (a short chunk, or the packed queries of a
  // small shared-prefix group): tile 1 is skipped and its S columns become a
  // second S buffer of tile 0, so the next tile's S = QK^T overlaps this tile's
  // softmax.
  constexpr bool single = SINGLE;
  // Columns of O go through the epilogues 32 at a time.  Drafted tokens roll those loops: a
  // CTA runs them once, so their instructions come from the second-level cache at best,
  // and under a full memory load the unrolled form spent 4 to 10 us on fetching itself
  // (64 trees of 16 over 4k keys, E4M3: 227 us unrolled, 196 rolled).  The long passes of
  // the plain two-tile kernel keep them unrolled: rolled, its main loop came out of the
  // compiler 6 % slower (2048 queries over 131072 keys, 7.38 -> 7.85 ms with the decode).
  constexpr int kRoll = TREE || SINGLE ? 1 : D / 32;
  // TREE, item with queries in query tile 0 only (row word 6): both softmax groups work
  // on that tile, group t on K tiles t, t + 2, ... with an O of its own, and the two are
  // merged at the end.  (One group alone takes ~3200 cycles per K tile, exponentials,
  // packing and tensor-memory round trips in series, where the K/V bytes of a tile
  // arrive in 2600 over a bf16 cache and 1300 over an E4M3 one.)
  const bool dual = TREE && w1.z != 0;
  const int ahead = dual ? 2 : 1;  // K tiles go out this many before their V tile

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    // full: the copy's bytes, or over an FP8 cache the widening warp's arrival
    for (int s = 0; s < RK; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < RV; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 128);
      mbar_init(o_full + s, 1);
    }
    mbar_init(mma_done, 1);
    mbar_init(s_free, 4);  // one arrival per softmax warp of the tile that read S
    mbar_init(q_conv, (SINGLE ? 1 : 2) * 128);
    if (FP8) {
      for (int s = 0; s < RK; ++s) mbar_init(code_k + s, 1);
      for (int s = 0; s < RV; ++s) mbar_init(code_v + s, 1);
    }
    *abort_flag = 0;
    *nonfinite = 0;
    *mask_at = (uint64_t)(uint32_t)w3.y | ((uint64_t)(uint32_t)w3.z << 32);
    *wait_limit = p.wait_ns;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k.box128);
    prefetch_tensormap(&tm_v.box128);
    prefetch_tensormap(&tm_o);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int k_issued = 0, v_issued = 0;
    if (n_tiles > 0) {
      // bf16 cache: when the table gives the slot of a first K tile that lies inside
      // one segment, that tile goes with the query tiles, ahead of any table lookup
      // (a stage of the fresh ring is free)
      const bool k0_early = !FP8 && w3.x >= 0 && p.withhold_tile != 0;
      if (lane == 0) {
        const int q_tiles = single || dual ? 1 : 2;
        mbar_expect_tx(q_full, q_tiles * TILE);
        for (int t = 0; t < q_tiles; ++t)
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(sQ + t * QSTRIDE + h * kHalfBytes, &tm_q, q_full, 64 * h, g * p.group,
                        tok0 + q0 + t * p.qpt);
        if (k0_early) {
          mbar_expect_tx(k_full, TILE);
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(sK + h * kHalfBytes, &tm_k.box128, k_full, 64 * h, g, w3.x);
        }
      }
      // The segment that the last tile inside one segment lay in: key after it, first slot
      // minus first key.  Long segments need no other lookup: two compares a tile (a search
      // in the window below for every tile slowed one-tile items by 2 %).
      const int seg_end = w1.w;
      int seg0 = w2.w;
      const int key0 = __ldg(p.tab.seg_kstart + seg0);
      int cur_last = key0 + __ldg(p.tab.seg_len + seg0);
      int cur_off = __ldg(p.tab.seg_start + seg0) - key0;
      // The request's segments from there on, 32 at a time, one per lane, once a tile
      // leaves that segment (loaded together: walking the arrays key by key is a chain of
      // dependent loads, microseconds for a tile across a segment boundary).  Lane l:
      // segment seg0 + l.
      bool window = false;
      int seg_key, seg_off;  // first key; first slot minus first key
      int seg_last;          // key after the last one
      auto load_segments = [&]() {
        const int s = seg0 + lane;
        const bool live = s < seg_end;
        seg_key = live ? __ldg(p.tab.seg_kstart + s) : 0x7fffffff;
        seg_off = live ? __ldg(p.tab.seg_start + s) - seg_key : 0;
        seg_last = live ? seg_key + __ldg(p.tab.seg_len + s) : 0x7fffffff;
      };
      // lane of the segment that holds key j (the last one that starts at or before it)
      auto segment_of = [&](int j) -> int {
        for (;;) {
          const uint32_t before = __ballot_sync(0xffffffffu, seg_key <= j);
          const int l = 31 - __clz(before);
          if (l < 31 || seg0 + 32 >= seg_end) return max(l, 0);
          seg0 += 31;  // the window's last segment, and those after it
          load_segments();
        }
      };
      // Pool rows of K tile i: lane l holds logical keys 4l .. 4l + 3 (keys past the
      // request are clamped to its last key).  Most tiles are 128 consecutive pool
      // slots (segments are long): one tiled box per 64-column half.  In a tile that
      // straddles a segment boundary or the end of the request, every aligned group of 32
      // or 8 keys in consecutive slots is a box of its own and only the rest is gathered
      // four rows at a time (a gather of 4 rows costs the TMA engine as much as a box of
      // 32: gathering all 128 rows took 2.3 us, 16 copies where there were 64 take 0.6).
      // Drafted tokens: rows past the request are not loaded (clean_v).  Tiles are
      // visited in increasing order (the segment cursor only moves on).
      enum { kNothing = -1, kGather = 0, kBox8 = 1, kBox32 = 2 };
      struct TileRows {
        int rows[4];
        int slot0;   // contiguous: the tile's first slot; otherwise this lane's
        int kind;    // not contiguous: what this lane loads
        int count;   // rows loaded
        bool contiguous;
      };
      auto tile_rows = [&](int i, TileRows& tr) {
        // the usual case: all 128 keys inside one segment, i.e. 128 consecutive pool
        // slots, the same on every lane
        const int j0 = (kt0 + i) * kTileKeys;
        tr.count = kTileKeys;
        if (j0 + kTileKeys <= cur_last) {
          tr.slot0 = j0 + cur_off;
          tr.contiguous = true;
          return;
        }
        if (!window) load_segments();
        window = true;
        int l = segment_of(j0);
        int off = __shfl_sync(0xffffffffu, seg_off, l);
        const int end = __shfl_sync(0xffffffffu, seg_last, l);
        if (j0 + kTileKeys <= end) {
          cur_last = end;
          cur_off = off;
          tr.slot0 = j0 + off;
          tr.contiguous = true;
          return;
        }
        const int last = min(j0 + kTileKeys, k_len) - 1;
        int key[4], at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          key[e] = min(j0 + 4 * lane + e, last);
          at[e] = off;
        }
        // the segments that begin inside the tile
        for (;;) {
          if (++l == 32) {
            if (seg0 + 32 >= seg_end) break;
            seg0 += 31;  // keep the window's last segment: the next tile may begin in it
            load_segments();
            l = 1;
          }
          const int first = __shfl_sync(0xffffffffu, seg_key, l);
          if (first > last) break;
          off = __shfl_sync(0xffffffffu, seg_off, l);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key[e] >= first) at[e] = off;
        }
        bool four = true;
        tr.slot0 = key[0] + at[0];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int slot = key[e] + at[e];
          tr.rows[e] = slot * p.kv_heads + g;
          four &= slot == tr.slot0 + e;
        }
        // lanes whose rows are consecutive slots, and follow those of the lane before
        const uint32_t runs = __ballot_sync(0xffffffffu, four);
        const int before = __shfl_up_sync(0xffffffffu, tr.slot0, 1);
        const uint32_t links = __ballot_sync(0xffffffffu, tr.slot0 == before + 4);
        tr.contiguous = runs == 0xffffffffu && (links | 1u) == 0xffffffffu;
        if (tr.contiguous) {
          tr.slot0 = __shfl_sync(0xffffffffu, tr.slot0, 0);
          return;
        }
        const uint32_t o = runs >> (lane & ~7) & 0xffu, ol = links >> (lane & ~7) & 0xfeu;
        const uint32_t w = runs >> (lane & ~1) & 3u, wl = links >> (lane & ~1) & 2u;
        if (o == 0xffu && ol == 0xfeu)
          tr.kind = (lane & 7) == 0 ? kBox32 : kNothing;
        else if (w == 3u && wl == 2u)
          tr.kind = (lane & 1) == 0 ? kBox8 : kNothing;
        else
          tr.kind = kGather;
        if (TREE) {
          const int left = k_len - j0;
          if (4 * lane >= left) tr.kind = kNothing;
          tr.count = min(kTileKeys, (left + 3) & ~3);
        }
      };
      // the rows of a tile, `bytes` each, `cols` columns per box and `panels` of them.  A
      // contiguous tile has a path of its own: tested inside the panel loop, with the
      // warp's step before it, long one-tile items took 3 % more.
      auto load_rows = [&](const TileRows& tr, uint8_t* dst, const PoolMaps& map, uint64_t* bar,
                           int cols, int panels, int bytes) {
        if (tr.contiguous) {
          if (lane == 0) {
            mbar_expect_tx(bar, kTileKeys * panels * bytes);
#pragma unroll
            for (int h = 0; h < panels; ++h)
              tma_load_3d(dst + h * kHalfBytes, &map.box128, bar, cols * h, g, tr.slot0);
          }
          return;
        }
        if (lane == 0) mbar_expect_tx(bar, tr.count * panels * bytes);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < panels; ++h) {
          uint8_t* at = dst + h * kHalfBytes + lane * 4 * bytes;
          if (tr.kind == kBox32) {
            tma_load_3d(at, &map.box32, bar, cols * h, g, tr.slot0);
          } else if (tr.kind == kBox8) {
            tma_load_3d(at, &map.box8, bar, cols * h, g, tr.slot0);
          } else if (tr.kind == kGather) {
            tma_gather4(at, &map.row, bar, cols * h, tr.rows[0], tr.rows[1], tr.rows[2], tr.rows[3]);
          }
        }
      };
      // bf16: 64-column panels in the swizzled layout; FP8: raw code rows, no swizzle
      auto load_tile = [&](const TileRows& tr, uint8_t* dst, const PoolMaps& map, uint64_t* bar) {
        load_rows(tr, dst, map, bar, 64, HALVES, 128);
      };
      auto load_codes = [&](const TileRows& tr, uint8_t* dst, const PoolMaps& map, uint64_t* bar) {
        load_rows(tr, dst, map, bar, 0, 1, D);
      };
      auto load_k = [&](int i, const TileRows& tr) -> bool {
        // stall test: stop loading here, as a copy that never lands would; the
        // consumers' bounded waits then give up and the CTA drains and exits
        if (i == p.withhold_tile) return false;
        const int st = i % RK;
        if (!__all_sync(0xffffffffu, mbar_wait(k_empty + st, ((i / RK) & 1) ^ 1, abort_flag,
                                               wait_limit, true)))
          return false;
        if (FP8)  // codes into the slot's second half, widened there by the last warps
          load_codes(tr, sK + st * TILE + TILE / 2, tm_k, code_k + st);
        else
          load_tile(tr, sK + st * TILE, tm_k, k_full + st);
        ++k_issued;
        return true;
      };
      auto load_v = [&](int i, const TileRows& tr) -> bool {
        const int st = i % RV;
        if (!__all_sync(0xffffffffu, mbar_wait(v_empty + st, ((i / RV) & 1) ^ 1, abort_flag,
                                               wait_limit, true)))
          return false;
        if (FP8)
          load_codes(tr, sV + st * TILE + TILE / 2, tm_v, code_v + st);
        else
          load_tile(tr, sV + st * TILE, tm_v, v_full + st);
        ++v_issued;
        return true;
      };
      // K tile i + 1 (dual: i + 2) before V tile i: the MMA warp takes them in that order
      TileRows cur, nxt, far;
      tile_rows(0, cur);
      if (k0_early) ++k_issued;
      bool run = k0_early || load_k(0, cur);
      if (dual && n_tiles > 1) {
        tile_rows(1, nxt);
        run = run && load_k(1, nxt);
      }
      for (int i = 0; run && i < n_tiles; ++i) {
        if (i + ahead < n_tiles) {
          tile_rows(i + ahead, far);
          if (!(run = load_k(i + ahead, far))) break;
        }
        if (!(run = load_v(i, cur))) break;
        cur = dual ? nxt : far;
        nxt = far;
      }
      // never leave the CTA with copies in flight (the copies' own barriers:
      // over an FP8 cache the slots' full barriers wait for the widening threads too)
      for (int s = 0; s < RK; ++s)
        if (k_issued > s) {
          const int last = s + RK * ((k_issued - 1 - s) / RK);
          mbar_wait((FP8 ? code_k : k_full) + s, (last / RK) & 1, nullptr, wait_limit);
        }
      for (int s = 0; s < RV; ++s)
        if (v_issued > s) {
          const int last = s + RV * ((v_issued - 1 - s) / RV);
          mbar_wait((FP8 ? code_v : v_full) + s, (last / RV) & 1, nullptr, wait_limit);
        }
      if (lane == 0) mbar_wait(q_full, 0, nullptr, wait_limit);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the issue loop on warp-uniform values; one elected lane
    // executes each tcgen05.mma / commit.
    if (n_tiles > 0) {
      // The issue loop is one warp sharing its sub-partition with two softmax warps,
      // so every instruction on it adds latency to the period: a complete phase is
      // taken on the first try (uniform across the warp, no vote), and several
      // barriers get independent first tries whose latencies overlap; the bounded
      // wait runs only when a phase is not complete yet.
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(smem_u32(bar), parity)) return true;
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, wait_limit, true)) != 0;
      };
      auto ready = [&](uint64_t* bar, uint32_t parity) { return mbar_try_wait(smem_u32(bar), parity); };
      const uint32_t idesc_qk =
          FP8 ? idesc_f16_f32(128, 128, false) : idesc_bf16_f32(128, 128, false);
      const uint32_t idesc_pv = FP8 ? idesc_f16_f32(128, D, true) : idesc_bf16_f32(128, D, true);
      const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK), v_addr = smem_u32(sV);
      const uint32_t tS0 = tmem + 256, tO0 = tmem, tP0 = tmem + 384;
      // S buffer `sb` = Q tile `qt` . K stage `st`^T;  O tile `ot` += P (in S buffer `sb`) . V stage `st`
      // Shared-memory descriptors are built once: a ring stage or P tile moves the
      // start address (16-byte units, the low 14 bits) by a multiple of its size,
      // and each 16-deep K step by a constant.  Building them per MMA inside the
      // issue loop measured ~1.8x slower MMA issue than the tensor core's rate.
      const uint64_t dq = sdesc_sw128(q_addr, 16, 1024), dk = sdesc_sw128(k_addr, 16, 1024);
      const uint64_t dv = sdesc_sw128(v_addr, kHalfBytes, 1024);
      constexpr uint32_t kTileU = TILE >> 4;
      // K-step k of a K-major operand: panel k / 4, 32 bytes per step inside it
      auto kstep = [](int k) -> uint32_t { return ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4; };
      // S buffer `sb` = Q tile `qt` . K stage `st`^T;  O tile `ot` += P (in S buffer `sb`) . V stage `st`
      auto issue_qk = [&](int qt, int sb, int st) {
        const uint64_t a0 = dq + qt * kTileU, b0 = dk + st * kTileU;
        const uint32_t d = tS0 + 128 * sb;
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k)
          mma_ss_warp(d, a0 + kstep(k), b0 + kstep(k), idesc_qk, k > 0 ? 1u : 0u);
      };
      // one tile: O += P (region `sb`, columns [128 + 64 sb, 192 + 64 sb)) . V stage `st`
      auto issue_pv = [&](int ot, int sb, int st, bool acc) {
        const uint64_t b0 = dv + st * kTileU;
        const uint32_t d = tO0 + 128 * ot, a = tmem + 128 + 64 * sb;
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k)
          mma_ts_warp(d, a + 8 * k, b0 + ((k * 2048) >> 4), idesc_pv, (acc || k > 0) ? 1u : 0u);
      };
      // two tiles: S = Q tile `qt` . K stage `st`^T into the shared S buffer (SS);
      // O tile `ot` += P tile `ot` (its own tensor-memory columns) . V stage `st` (TS)
      auto issue_qk_t = [&](int qt, int st) {
        const uint64_t a0 = dq + qt * kTileU, b0 = dk + st * kTileU;
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k)
          mma_ss_warp(tS0, a0 + kstep(k), b0 + kstep(k), idesc_qk, k > 0 ? 1u : 0u);
      };
      auto issue_pv_s = [&](int ot, int st, bool acc) {
        const uint64_t b0 = dv + st * kTileU;
        const uint32_t d = tO0 + 128 * ot, a = tP0 + 64 * ot;
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k)
          mma_ts_warp(d, a + 8 * k, b0 + ((k * 2048) >> 4), idesc_pv, (acc || k > 0) ? 1u : 0u);
      };
      // FP8: the softmax threads convert the query tiles to f16 in place first
      bool ok = wait_all(FP8 ? q_conv : q_full, 0) && wait_all(k_full + 0, 0);
      if (single) {
        // one query tile, S double-buffered: K tile i uses S buffer and P region i & 1.
        // While the softmax works on buffer i & 1, S of tile i + 1 is already in the
        // other one; right after PV(i), S of tile i + 2 goes into buffer i & 1 (the PV
        // reads P region i & 1, not the S columns).  Tensor-core operations of one CTA
        // run in issue order, so S of tile i + 2 being complete also means PV(i) is, and
        // the softmax may then overwrite P region i & 1.
        if (ok) {
          tc_fence_after();
          issue_qk(0, 0, 0);
          mma_commit_warp(s_full + 0);
          mma_commit_warp(k_empty + 0);
        }
        if (ok && n_tiles > 1 && (ok = wait_all(k_full + 1, 0))) {
          tc_fence_after();
          issue_qk(0, 1, 1);
          mma_commit_warp(s_full + 1);
          mma_commit_warp(k_empty + 1);
        }
        // S buffer of tile i: i & 1; its ring stages: i % RK, i % RV
        for (int i = 0; ok && i < n_tiles; ++i) {
          const int b = i & 1, vs = i % RV;
          const uint32_t ph = (i >> 1) & 1;
          if (!(ok = wait_all(v_full + vs, (i / RV) & 1))) break;
          if (!(ok = wait_all(p_full + b, ph))) break;
          tc_fence_after();
          issue_pv(0, b, vs, i > 0);
          mma_commit_warp(o_full + 0);
          mma_commit_warp(v_empty + vs);
          if (i + 2 < n_tiles) {
            const int ks = (i + 2) % RK;
            if (!(ok = wait_all(k_full + ks, ((i + 2) / RK) & 1)))
              break;
            tc_fence_after();
            issue_qk(0, b, ks);
            mma_commit_warp(s_full + b);
            mma_commit_warp(k_empty + ks);
          }
        }
      } else if (dual) {
        // One query tile, two softmax groups, one S buffer.  Use i of the buffer is QK of
        // K tile i, for group i & 1; it may start once the other group has read use i - 1
        // (completion i - 1 of s_free).  Order: QK(i + 2), PV(i), with P and O of the group.
        for (int i = 0; ok && i < 2 && i < n_tiles; ++i) {
          if (i > 0 && !(ok = wait_all(k_full + i, 0) && wait_all(s_free, 0))) break;
          tc_fence_after();
          issue_qk_t(0, i);
          mma_commit_warp(s_full + i);
          mma_commit_warp(k_empty + i);
        }
        for (int i = 0; ok && i < n_tiles; ++i) {
          const int g2 = i & 1, st = i % RV;
          if (i + 2 < n_tiles) {
            const int st2 = (i + 2) % RK;
            if (!(ok = wait_all(k_full + st2, ((i + 2) / RK) & 1) && wait_all(s_free, (i + 1) & 1)))
              break;
            tc_fence_after();
            issue_qk_t(0, st2);
            mma_commit_warp(s_full + g2);
            mma_commit_warp(k_empty + st2);
          }
          if (!(ok = wait_all(v_full + st, (i / RV) & 1) && wait_all(p_full + g2, (i >> 1) & 1)))
            break;
          tc_fence_after();
          issue_pv_s(g2, st, i > 1);
          mma_commit_warp(o_full + g2);
          mma_commit_warp(v_empty + st);
        }
      } else {
        // Two tiles, one S buffer.  Use u of the buffer is QK of K tile u / 2 for
        // query tile u % 2; it may start once the softmax has read use u - 1
        // (completion u - 1 of s_free).  Per K tile i the order is
        //   QK_0(i + 1), PV_0(i), QK_1(i + 1), PV_1(i)
        // so the S of a query tile's next K tile is ready when its softmax
        // finishes the current one.
        if (ok) {
          tc_fence_after();
          issue_qk_t(0, 0);
          mma_commit_warp(s_full + 0);
        }
        if (ok && (ok = wait_all(s_free, 0))) {
          tc_fence_after();
          issue_qk_t(1, 0);
          mma_commit_warp(s_full + 1);
          mma_commit_warp(k_empty + 0);
        }
        for (int i = 0; ok && i < n_tiles; ++i) {
          const int st = i % RV;  // V stage of K tile i
          const uint32_t ph = (i / RV) & 1;
          const bool more = i + 1 < n_tiles;
          const int st1 = (i + 1) % RK;  // K stage of K tile i + 1
          const uint32_t ph1 = ((i + 1) / RK) & 1;
          if (more) {
            // use 2i + 2 waits for completion 2i + 1 (tile 1 read S of K tile i)
            if (!(ready(k_full + st1, ph1) & ready(s_free, 1)) &&
                !(ok = wait_all(k_full + st1, ph1) && wait_all(s_free, 1)))
              break;
            tc_fence_after();
            issue_qk_t(0, st1);
            mma_commit_warp(s_full + 0);
          }
          if (!(ready(v_full + st, ph) & ready(p_full + 0, i & 1)) &&
              !(ok = wait_all(v_full + st, ph) && wait_all(p_full + 0, i & 1)))
            break;
          tc_fence_after();
          issue_pv_s(0, st, i > 0);
          mma_commit_warp(o_full + 0);
          if (more) {
            // use 2i + 3 waits for completion 2i + 2 (tile 0 read S of K tile i + 1)
            if (!(ok = wait_all(s_free, 0)))
              break;
            tc_fence_after();
            issue_qk_t(1, st1);
            mma_commit_warp(s_full + 1);
            mma_commit_warp(k_empty + st1);
          }
          if (!(ok = wait_all(p_full + 1, i & 1))) break;
          tc_fence_after();
          issue_pv_s(1, st, i > 0);
          mma_commit_warp(o_full + 1);
          mma_commit_warp(v_empty + st);
        }
      }
      // all MMAs finished before tensor memory is released
      mma_commit_warp(mma_done);
      mbar_wait(mma_done, 0, nullptr, wait_limit);
    }
    __syncwarp();
  } else if (FP8 && warp >= kConvWarp0) {
    // ------------------------------------------------------------ FP8 code widening
    // E4M3 tile -> f16 K (V) ring slot, then make the generic-proxy writes
    // visible to the tensor cores before signalling the ring slot full.
    const bool is_k = warp == kConvWarp0;
    uint8_t* ring = is_k ? sK : sV;
    uint64_t* landed = is_k ? code_k : code_v;
    uint64_t* full = is_k ? k_full : v_full;
    const int depth = is_k ? RK : RV;
    for (int i = 0, st = 0, ph = 0; i < n_tiles; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(landed + st, ph, abort_flag, wait_limit))) break;
      widen_tile<D>(ring + st * TILE, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + st);
      if (++st == depth) {
        st = 0;
        ph ^= 1;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int t = (warp - 2) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int tq = dual ? 0 : t;  // query tile of this group's rows
    const int qi = q0 + tq * p.qpt + row / p.group;
    const int head = g * p.group + row % p.group;
    const bool row_valid = qi < q_len;
    const int prior = k_len - q_len;  // TREE: keys before the drafted ones
    // TREE: this row's mask row.  Its address comes from shared memory where it is needed:
    // in registers across the K tiles it would cost spills.
    auto mask_row = [&]() -> const uint32_t* {
      return p.mask_base + *mask_at + (int64_t)qi * ((q_len + 31) >> 5);
    };
    if (TREE && row_valid) prefetch_global(mask_row());
    // TREE: which of the 32 keys from drafted key `at` on this row sees (at < 0: cached
    // keys, all seen, come first)
    auto mask_word = [&](const uint32_t* mrow, int at) -> uint32_t {
      if (at <= -32) return 0xffffffffu;
      if (!row_valid) return 0u;
      const int words = (q_len + 31) >> 5;
      if (at < 0) return (__ldg(mrow) << -at) | ((1u << -at) - 1u);
      const int w = at >> 5;
      const uint32_t lo = w < words ? __ldg(mrow + w) : 0u;
      const uint32_t hi = w + 1 < words ? __ldg(mrow + w + 1) : 0u;
      return __funnelshift_r(lo, hi, at & 31);
    };
    const int vis = TREE ? prior : p.causal ? min(k_len, k_len - q_len + qi + 1) : k_len;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t tS = lane_base + 256 + 128 * t;  // S buffer of the current K tile (SINGLE)
    if (QT) tS = lane_base + 256;             // two tiles: the shared S buffer
    const uint32_t tO = lane_base + 128 * t;
    // P of the current K tile: two tiles, this tile's region; one tile, the region of
    // the current S buffer (set per K tile)
    uint32_t tP = lane_base + 384 + 64 * t;
    // FP8: scores are q . code * k_scale, so the K scale joins the softmax scale
    const float sl2 = FP8 ? p.scale_log2 * __ldg(p.k_scale + g) : p.scale_log2;
    const int my_tiles = dual ? (n_tiles - t + 1) >> 1 : n_tiles;  // K tiles of this group
    float m_ref = -INFINITY;  // raw score units
    float l = 0.f;
    // a row that saw a NaN score has a NaN sum, which its lse shows (drafted tokens)
    auto has_keys = [](float sum) { return TREE ? sum != 0.f : sum > 0.f; };
    bool ok = true;
    if (n_tiles > 0 && FP8) {
      // FP8 cache: this thread's query row of tile t, bf16 -> f16 in place (exact
      // for |q| < 65504), so that both MMA operands are f16.  Visiting chunk
      // c ^ (row & 7), the place of the row's logical chunk c, spreads a warp's
      // 32 rows over all shared-memory banks.
      ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, abort_flag, wait_limit));
      if (ok) {
        if (!dual || t == 0) {
#pragma unroll 1
          for (int h = 0; h < HALVES; ++h)
#pragma unroll 4
            for (int c = 0; c < 8; ++c) {
              uint4* chunk = reinterpret_cast<uint4*>(sQ + t * QSTRIDE + h * kHalfBytes +
                                                      row * 128 + ((c ^ (row & 7)) << 4));
              uint4 v = *chunk;
              bf16x8_to_f16x8(v);
              *chunk = v;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_conv);
      }
    }
    // One tile of the online softmax.  `masked`: some row of the warp must not
    // see some key of the tile (causal diagonal, end of the request); the mask
    // is applied to the registers, so other tiles never compare per element.
    // K tile i is this group's j-th (i = j unless dual).
    auto softmax_tile = [&](int i, int j, bool masked) -> bool {
      auto f = [](uint32_t bits) { return __uint_as_float(bits); };
      // TREE: the tile's mask words, before the S row takes its 128 registers (bf16) or
      // where they are used (FP8): the order that leaves the loop without spills
      uint32_t words[4] = {0u, 0u, 0u, 0u};
      auto load_words = [&]() {
        const uint32_t* mrow = mask_row();
#pragma unroll
        for (int c = 0; c < 4; ++c) words[c] = mask_word(mrow, (kt0 + i) * kTileKeys + 32 * c - prior);
      };
      if (TREE && !FP8 && masked) load_words();
      // the whole S row in registers: one round trip to tensor memory
      uint32_t sv[4][32];
      tmem_ld128(tS, sv);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld(sv[c]);
      if (QT) {
        // the shared S buffer is free for the other tile's QK
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
      }
      if (masked) {
        const int kb = (kt0 + i) * kTileKeys;
        if (TREE && FP8) load_words();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t word = TREE ? words[c] : 0u;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const bool hide = TREE ? !((word >> e) & 1u) : kb + 32 * c + e >= vis;
            if (hide) sv[c][e] = 0xff800000u;  // -inf
          }
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) mx[c] = max3(mx[c], f(sv[c][e]), f(sv[c][e + 1]));
      const float row_max = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
      const float m_new = fmaxf(m_ref, row_max);
      float alpha = 1.f;
      bool rescale = false;
      if (m_ref == -INFINITY) {
        m_ref = m_new;  // nothing accumulated yet for this row (or only zeros)
      } else if ((m_new - m_ref) * sl2 > kRescaleLog2) {
        alpha = ex2((m_ref - m_new) * sl2);
        m_ref = m_new;
        rescale = true;
      }
      const float base = m_ref == -INFINITY ? 0.f : m_ref * sl2;
      // P = 2^(s*scale*log2e - base), packed in pairs: bf16, or f16 over an FP8 cache (V is
      // widened to f16 there).  The one rounding of a weight, by at most 2^-8 or 2^-11 of
      // it, is the price of the tensor cores' 16-bit operand; the sum l takes the unrounded
      // ones.  Two tiles: f32x2 pairs for the scale-and-subtract and the sums (fewer
      // instructions per score); the one-tile kernel keeps scalar arithmetic, whose register
      // allocation does not spill.
      uint64_t ls = f2_pack(0.f, 0.f);
      float ls0 = 0.f, ls1 = 0.f;
      const uint64_t sl2x2 = f2_pack(sl2, sl2), nbase2 = f2_pack(-base, -base);
      uint32_t pk[4][16];
      // two tiles: P(i) replaces P(i - 1) in this tile's tensor-memory columns once
      // PV(i - 1) has read it (complete by now as a rule: it was issued when this
      // tile's S was)
      bool waited = false;
      if (QT && j > 0) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait(o_full + t, (j - 1) & 1, abort_flag, wait_limit, true)))
          return false;
        tc_fence_after();
        waited = true;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float pa, pb;
          if constexpr (!QT) {
            pa = ex2(fmaf(f(sv[c][2 * e]), sl2, -base));
            pb = ex2(fmaf(f(sv[c][2 * e + 1]), sl2, -base));
            ls0 += pa;
            ls1 += pb;
          } else {
            float xa, xb;
            f2_unpack(f2_fma(f2_pack(f(sv[c][2 * e]), f(sv[c][2 * e + 1])), sl2x2, nbase2), xa, xb);
            pa = ex2(xa);
            pb = ex2(xb);
            ls = f2_add(ls, f2_pack(pa, pb));
          }
          pk[c][e] = FP8 ? pack_f16x2(pa, pb) : pack_bf16(pa, pb);
        }
      }
      // 128 keys as 64 columns of 2 (the tensor-memory A-operand layout), one store
      tmem_st64(tP, pk);
      if constexpr (QT) f2_unpack(ls, ls0, ls1);
      l = l * alpha + (ls0 + ls1);
      if (__any_sync(0xffffffffu, rescale)) {
        // O_t holds PV up to this group's tile j - 1; rescale it in place once that is complete
        if (!waited &&
            !__all_sync(0xffffffffu, mbar_wait(o_full + t, (j - 1) & 1, abort_flag, wait_limit)))
          return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(tO + 32 * c, o);
        }
      }
      return true;
    };
    // A warp whose 32 rows hold no query (past the end of the chunk) only keeps
    // step with the barriers: its P rows feed only output rows nobody reads.
    const bool warp_live = __any_sync(0xffffffffu, row_valid);
    // One tile: before P of the last K tile n - 1 is signalled, PV(n - 2) must be
    // complete.  The S of tile n - 1 proves only PV(n - 3), and once P(n - 1) is
    // signalled PV(n - 1) may complete at any time; a later wait for PV(n - 2) could
    // then meet o_full at completion n, whose parity is that of n - 2, and wait for
    // a completion that never comes.  Confirmed here, o_full is at completion n - 1
    // or n when the epilogue waits for PV(n - 1), which one parity wait tells apart.
    auto last_pv_order = [&](int i) -> bool {
      if (!single || i != n_tiles - 1 || i == 0) return true;
      return __all_sync(0xffffffffu,
                        mbar_wait(o_full + t, (i - 1) & 1, abort_flag, wait_limit)) != 0;
    };
    // TREE, tile with drafted keys: V row `row` of the tile, when it is a drafted key's,
    // gets zeros for values that are not finite, and is all zeros past the last key.  Query tile 0's
    // threads (dual: the group that has the K tile) do it before they signal P; the PV of
    // query tile 1 is issued after tile 0's.
    auto clean_v = [&](int i) -> bool {
      const int sv = i % RV;
      if (!__all_sync(0xffffffffu, mbar_wait(v_full + sv, (i / RV) & 1, abort_flag, wait_limit)))
        return false;
      const int key = (kt0 + i) * kTileKeys + row;
      if (key < prior) return true;
      if (key >= k_len) {  // a row past the request: whatever shared memory held
#pragma unroll 1
        for (int h = 0; h < HALVES; ++h)
#pragma unroll 2
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(sV + sv * TILE + h * kHalfBytes + row * 128 +
                                      ((c ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        return true;
      }
      constexpr uint32_t kExp = FP8 ? 0x7c00u : 0x7f80u;  // f16 (widened) or bf16
      bool found = false;
#pragma unroll 1
      for (int h = 0; h < HALVES; ++h)
#pragma unroll 2
        for (int c = 0; c < 8; ++c) {
          uint32_t* w = reinterpret_cast<uint32_t*>(sV + sv * TILE + h * kHalfBytes + row * 128 +
                                                    ((c ^ (row & 7)) << 4));
          const uint4 v = *reinterpret_cast<const uint4*>(w);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool lo = (x[e] & kExp) == kExp, hi = (x[e] & (kExp << 16)) == (kExp << 16);
            if (lo || hi) {
              w[e] = (lo ? 0u : x[e] & 0xffffu) | (hi ? 0u : x[e] & 0xffff0000u);
              found = true;
            }
          }
        }
      if (found) {
        *reinterpret_cast<volatile int*>(nonfinite) = 1;
        fence_proxy_async_smem();
      }
      return true;
    };
    // one K tile of softmax on S buffer sb (phase sph of its barriers)
    auto run_tile = [&](int i, int j, int sb, uint32_t sph) -> bool {
      if (single) {
        tS = lane_base + 256 + 128 * sb;
        tP = lane_base + 128 + 64 * sb;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(s_full + sb, sph, abort_flag, wait_limit, true)))
        return false;
      if (!warp_live) {
        if (QT) {
          // release S; arrive for P(i) only after PV(i - 1), so that these
          // arrivals never count towards the previous P
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
          if (j > 0 &&
              !__all_sync(0xffffffffu, mbar_wait(o_full + t, (j - 1) & 1, abort_flag, wait_limit)))
            return false;
        }
        if (!last_pv_order(i)) return false;
        if (TREE && tq == 0 && (kt0 + i + 1) * kTileKeys > prior && !clean_v(i)) return false;
        mbar_arrive(p_full + sb);
        return true;
      }
      tc_fence_after();
      const bool masked = __any_sync(0xffffffffu, (kt0 + i + 1) * kTileKeys > vis);
      if (!softmax_tile(i, j, masked)) return false;
      tmem_wait_st();
      if (!last_pv_order(i)) return false;
      if (TREE && tq == 0 && masked && !clean_v(i)) return false;
      tc_fence_before();
      mbar_arrive(p_full + sb);
      return true;
    };
    if (single) {
      // S buffers alternate; unrolled by two so each buffer's address is fixed
      for (int i = 0; ok && i < n_tiles; i += 2) {
        const uint32_t sph = (i >> 1) & 1;
        ok = run_tile(i, i, 0, sph);
        if (ok && i + 1 < n_tiles) ok = run_tile(i + 1, i + 1, 1, sph);
      }
    } else {
      for (int j = 0; ok && j < my_tiles; ++j)
        ok = run_tile(dual ? 2 * j + t : j, j, t, j & 1);
    }
    // order test (one tile): the last PV completes before this warp reaches the end
    // of the item
    if constexpr (SINGLE) {
      if (p.p_delay_ns > 0 && ok) __nanosleep(p.p_delay_ns);
    }
    // TREE, after some drafted V value was not finite: what this row sees of them is added
    // to O in tensor memory, as its product with a positive weight would be (a NaN or an
    // infinity).  32 columns at a time, every lane of the warp in step.
    auto add_nonfinite = [&]() {
      const uint32_t* mrow = mask_row();
      const int first = max(kt0 * kTileKeys - prior, 0);
      const int last = min((kt0 + n_tiles) * kTileKeys - prior, q_len);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * c, o);
        tmem_wait_ld(o);
#pragma unroll 1
        for (int j = first; j < last; ++j) {
          // dual: drafted keys in this group's K tiles
          if (dual && ((((prior + j) / kTileKeys) ^ kt0 ^ t) & 1)) continue;
          const bool seen = mask_word(mrow, j) & 1u;
          const int64_t at =
              ((int64_t)__ldg(p.draft_slot + tok0 + j) * p.kv_heads + g) * D + 32 * c;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x = 0.f;
            if (FP8) {
              if ((static_cast<const uint8_t*>(p.v_pool)[at + e] & 0x7f) == 0x7f) x = NAN;
            } else {
              const uint32_t b = static_cast<const uint16_t*>(p.v_pool)[at + e];
              if ((b & 0x7f80) == 0x7f80) x = __uint_as_float(b << 16);
            }
            if (seen && x != 0.f) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
          }
        }
        tmem_st32(tO + 32 * c, o);
      }
      tmem_wait_st();
    };
    // dual: weights of the two groups' O, which group 0 adds up; group 1's (m, l) wait in
    // shared memory (in the K ring, which is free then)
    float w_own = 1.f, w_other = 0.f;
    float2* other_ml = reinterpret_cast<float2*>(sK);
    // 32 columns of this row's O (fp32).
    auto load_o = [&](int c, uint32_t (&o)[32]) {
      if (n_tiles == 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
        return;
      }
      tmem_ld32(tO + 32 * c, o);
      tmem_wait_ld(o);
      // the other group's rows lie in the same tensor-memory lanes, 128 columns on
      if (TREE && __any_sync(0xffffffffu, w_other != 0.f)) {
        uint32_t x[32];
        tmem_ld32(lane_base + 128 + 32 * c, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float y = __uint_as_float(o[e]) * w_own;
          if (w_other != 0.f) y = fmaf(__uint_as_float(x[e]), w_other, y);
          o[e] = __float_as_uint(y);
        }
      }
    };
    // before the first load_o
    auto open_o = [&]() {
      tc_fence_after();
      if (TREE && n_tiles > 0 && *reinterpret_cast<volatile int*>(nonfinite) != 0) add_nonfinite();
    };
    // 16-byte chunk k (eight columns) of 32 loaded ones, scaled, as bf16
    auto pack_o = [&](const uint32_t (&o)[32], int k, float inv) {
      auto f = [&](int e) { return __uint_as_float(o[8 * k + e]) * inv; };
      return make_uint4(pack_bf16(f(0), f(1)), pack_bf16(f(2), f(3)), pack_bf16(f(4), f(5)),
                        pack_bf16(f(6), f(7)));
    };
    // PV complete up to tile n - 2 (two tiles: P(n - 1) was written after it; one
    // tile: confirmed before P(n - 1) was signalled), so o_full is at completion
    // n - 1 or n and a parity wait for PV(n - 1) is unambiguous
    if (ok && my_tiles > 0)
      ok = __all_sync(0xffffffffu,
                      mbar_wait(o_full + t, (my_tiles - 1) & 1, abort_flag, wait_limit));
    if (dual) {
      // Group 1 hands over its (m, l) and is done; its O stays in tensor memory, complete.
      // All of the item's QK are complete once its last PV is (QK of the last K tile is
      // issued before it), so the K ring is free.  Both groups meet at an AND of their
      // outcomes, so a give-up leaves no one waiting.
      if (t == 1 && ok && my_tiles > 0) {
        if (*reinterpret_cast<volatile int*>(nonfinite) != 0) {
          tc_fence_after();
          add_nonfinite();
        }
        other_ml[row] = make_float2(m_ref, l);
        tc_fence_before();
      }
      ok = named_barrier_and(4, 256, ok);
      tc_fence_after();
      if (t == 1) ok = false;  // nothing to write
      if (ok && n_tiles > 1) {
        const float2 ml = other_ml[row];
        const float top = fmaxf(m_ref, ml.x);
        // a group that saw no key has a zero O (and m = -inf): its weight must not be NaN
        w_own = m_ref == top ? 1.f : ex2((m_ref - top) * sl2);
        w_other = ml.x == top ? 1.f : ex2((ml.x - top) * sl2);
        l = l * w_own + ml.y * w_other;
        m_ref = top;
      }
    }
    if (!warp_live) ok = false;  // nothing to write
    // Results leave through shared memory so that whole rows are stored: a thread
    // owns one row, and its own 16-byte pieces of it would put every warp store on 32
    // different lines.  The tile's query region is free (the commit of the tile's
    // last PV covers every earlier MMA).  Each warp stages its 32 rows in a quarter of it
    // and copies rows out with consecutive lanes on consecutive 16-byte chunks; chunk c of
    // row-local r sits at ((c & ~7) | ((c ^ r) & 7)).
    uint8_t* stage_w = sQ + t * QSTRIDE + quad * (QSTRIDE / 4);
    auto swz = [](int c, int r) { return (c & ~7) | ((c ^ r) & 7); };
    if (ok && slot >= 0) {
      // piece of a split item (or of a shared-prefix pass): O / l and log2(sum of exp)
      // of this key range, for every row that holds a query; fp32 rows go out in passes
      // of 32 columns
      const float inv = has_keys(l) ? (FP8 ? __ldg(p.v_scale + g) : 1.f) / l : 0.f;
      const int64_t prow0 = (int64_t)slot * kItemRows + t * kTileRows + quad * 32;
      open_o();
#pragma unroll kRoll
      for (int pass = 0; pass < D / 32; ++pass) {
        uint32_t o[32];
        load_o(pass, o);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<float4*>(stage_w + lane * 128 + swz(c, lane) * 16) =
              make_float4(__uint_as_float(o[4 * c]) * inv, __uint_as_float(o[4 * c + 1]) * inv,
                          __uint_as_float(o[4 * c + 2]) * inv, __uint_as_float(o[4 * c + 3]) * inv);
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < 32; k += 4) {
          const int lr = k + lane / 8, c = lane % 8;
          const int qi_r = q0 + tq * p.qpt + (quad * 32 + lr) / p.group;
          if (qi_r < q_len)
            *reinterpret_cast<float4*>(p.part_o + (prow0 + lr) * D + pass * 32 + 4 * c) =
                *reinterpret_cast<const float4*>(stage_w + lr * 128 + swz(c, lr) * 16);
        }
        __syncwarp();
      }
      if (row_valid) p.part_lse[prow0 + lane] = has_keys(l) ? m_ref * sl2 + log2f(l) : -INFINITY;
    } else if (!TMA_OUT && ok) {
      // a pass whose pieces mostly write partials: rows staged per warp, copied out
      constexpr int CH = D / 8;    // 16-byte chunks of a bf16 row
      constexpr int RPI = 32 / CH; // rows per warp instruction of the copy
      const float inv = has_keys(l) ? (FP8 ? __ldg(p.v_scale + g) : 1.f) / l : 0.f;
      open_o();
#pragma unroll kRoll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        load_o(c, o);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(stage_w + lane * (D * 2) + swz(4 * c + k, lane) * 16) =
              pack_o(o, k, inv);
      }
      __syncwarp();
#pragma unroll 4
      for (int k = 0; k < 32; k += RPI) {
        const int lr = k + lane / CH, c = lane % CH;
        const int rr = quad * 32 + lr;
        const int qi_r = q0 + t * p.qpt + rr / p.group;
        if (qi_r < q_len)
          *reinterpret_cast<uint4*>(p.out + ((int64_t)(tok0 + qi_r) * p.q_heads + g * p.group +
                                             rr % p.group) * D + 8 * c) =
              *reinterpret_cast<const uint4*>(stage_w + lr * (D * 2) + swz(c, lr) * 16);
      }
      if (row_valid && p.lse)
        p.lse[(int64_t)(tok0 + qi) * p.q_heads + head] =
            has_keys(l) ? (m_ref * sl2 + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    if (TMA_OUT && slot < 0) {
      // Final bf16 output, staged in the tile's query region in the layout of the
      // queries' TMA box (64-column panels of 128-byte rows, chunk c of row r at
      // c ^ (r & 7)).  A full query tile then leaves in two TMA stores issued by one
      // thread (the rows of one tile are qpt consecutive tokens x G heads, the box of
      // the output map); a tile with fewer queries than qpt is copied out a row per
      // D / 8 lanes, since a box would reach into the next request's rows.  The
      // tile's four warps agree at a barrier (an AND of their outcomes) before
      // staging, so a give-up anywhere leaves no warp waiting at the second one.
      constexpr int CH = D / 8;    // 16-byte chunks of a bf16 row
      constexpr int RPI = 32 / CH; // rows per warp instruction of the copy
      uint8_t* stage_t = sQ + t * QSTRIDE;
      const bool full = q0 + (t + 1) * p.qpt <= q_len;
      const bool go = full ? named_barrier_and(2 + t, 128, ok) : ok;
      if (go) {
        const float inv = has_keys(l) ? (FP8 ? __ldg(p.v_scale + g) : 1.f) / l : 0.f;
        open_o();
#pragma unroll kRoll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          load_o(c, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int ch = 4 * c + k;  // logical 16-byte chunk of the row
            *reinterpret_cast<uint4*>(stage_t + (ch >> 3) * kHalfBytes + row * 128 +
                                      (((ch & 7) ^ (row & 7)) << 4)) = pack_o(o, k, inv);
          }
        }
        if (full) {
          fence_proxy_async_smem();
          named_barrier(2 + t, 128);
          if (quad == 0 && lane == 0) {
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_store_3d(&tm_o, stage_t + h * kHalfBytes, 64 * h, g * p.group,
                           tok0 + q0 + t * p.qpt);
            bulk_commit_group();
            bulk_wait_group_read0();  // the staging must be read before the CTA exits
          }
        } else {
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < 32; k += RPI) {
            const int rr = quad * 32 + k + lane / CH, c = lane % CH;
            const int qi_r = q0 + t * p.qpt + rr / p.group;
            if (qi_r < q_len)
              *reinterpret_cast<uint4*>(p.out + ((int64_t)(tok0 + qi_r) * p.q_heads + g * p.group +
                                                 rr % p.group) * D + 8 * c) =
                  *reinterpret_cast<const uint4*>(stage_t + (c >> 3) * kHalfBytes + rr * 128 +
                                                  (((c & 7) ^ (rr & 7)) << 4));
          }
        }
        if (row_valid && p.lse)
          p.lse[(int64_t)(tok0 + qi) * p.q_heads + head] =
              has_keys(l) ? (m_ref * sl2 + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(&g_device_error, 1);
}

// Combine the pieces of each split item: weights 2^(lse_j - max) on the pieces'
// normalised outputs.  One warp per row, each lane D/32 consecutive columns.
template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
  constexpr int PER = D / 32;
  const int4 m0 = p.tab.merge[2 * blockIdx.x], m1 = p.tab.merge[2 * blockIdx.x + 1];
  const int req = m0.x, g = m0.y, q0 = m0.z, slot0 = m0.w, parts = m1.x;
  const int tok0 = __ldg(p.tab.q_offsets + req);
  const int q_len = __ldg(p.tab.q_offsets + req + 1) - tok0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int row = blockIdx.y * 8 + warp; row < kItemRows; row += 8 * gridDim.y) {
    const int t = row / kTileRows, r = row % kTileRows;
    const int qi = q0 + t * p.qpt + r / p.group;
    if (qi >= q_len) continue;
    const int head = g * p.group + r % p.group;
    float M = -INFINITY;
    for (int j = 0; j < parts; ++j)
      M = fmaxf(M, p.part_lse[(int64_t)(slot0 + j) * kItemRows + row]);
    const float Mb = M == -INFINITY ? 0.f : M;
    float acc[PER], L = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int j = 0; j < parts; ++j) {
      const int64_t prow = (int64_t)(slot0 + j) * kItemRows + row;
      const float w = ptx::ex2(p.part_lse[prow] - Mb);
      L += w;
      const float* po = p.part_o + prow * D + lane * PER;
#pragma unroll
      for (int e = 0; e < PER; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(po + e);
        acc[e] += w * x.x;
        acc[e + 1] += w * x.y;
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    __nv_bfloat16* orow = p.out + ((int64_t)(tok0 + qi) * p.q_heads + head) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; e += 2)
      *reinterpret_cast<uint32_t*>(orow + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0)
      p.lse[(int64_t)(tok0 + qi) * p.q_heads + head] =
          L > 0.f ? (Mb + log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// bf16 maps are 128-byte swizzled (tensor-core operand layout); byte maps
// (E4M3 codes, staged for widening) are plain row-major.
bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, bool bytes = false) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
            const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool SINGLE, bool FP8, bool TMA_OUT, bool TREE>
int launch_items(const CUtensorMap& tq, const CUtensorMap& to, const PoolMaps& tk,
                 const PoolMaps& tv, const PrefillParams& p, int n, cudaStream_t stream) {
  constexpr size_t smem = prefill_smem_bytes<D, SINGLE>();
  if (cudaFuncSetAttribute(prefill_kernel<D, SINGLE, FP8, TMA_OUT, TREE>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SEG_ATTN_ERR_CUDA;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n);
  cfg.blockDim = dim3(cta_threads<SINGLE, FP8>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = early;
  cfg.numAttrs = TREE ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, prefill_kernel<D, SINGLE, FP8, TMA_OUT, TREE>, tq, to, tk, tv, p) ==
                 cudaSuccess
             ? SEG_ATTN_OK
             : SEG_ATTN_ERR_CUDA;
}

template <int D, bool FP8, bool TREE>
int launch_prefill_d(const PrefillLaunch& a, cudaStream_t stream) {
  const seg_attn_table_desc& d = *a.desc;
  const int group = d.q_heads / d.kv_heads;
  CUtensorMap tq, to;
  PoolMaps tk, tv;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)d.q_heads, (cuuint64_t)d.total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)d.q_heads * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)d.queries_per_tile};
    if (!encode(&tq, a.q, 3, dims, strides, box)) return SEG_ATTN_ERR_CUDA;
    // the output has the queries' shape: full query tiles leave by TMA stores of the
    // same boxes (a pass that only writes partials has no output: no store is issued)
    if (!encode(&to, a.out ? a.out : a.q, 3, dims, strides, box)) return SEG_ATTN_ERR_CUDA;
  }
  {
    const int64_t rows = d.num_slots * d.kv_heads;
    const bool empty = rows == 0 || d.total_k == 0;
    // bf16: 64-column boxes (one swizzle panel); FP8: whole D-byte code rows
    constexpr int kElem = FP8 ? 1 : 2;
    constexpr cuuint32_t kBoxCols = FP8 ? D : 64;
    const cuuint64_t dims[2] = {(cuuint64_t)D, empty ? 1ull : (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * kElem};
    const cuuint32_t box[2] = {kBoxCols, 1};
    // the same pools as [slots][kv heads][d]: consecutive slots of one head per box
    const cuuint64_t dims3[3] = {(cuuint64_t)D, (cuuint64_t)d.kv_heads,
                                 empty ? 1ull : (cuuint64_t)d.num_slots};
    const cuuint64_t strides3[2] = {(cuuint64_t)D * kElem, (cuuint64_t)d.kv_heads * D * kElem};
    auto pool = [&](PoolMaps& m, const void* base) {
      if (!encode(&m.row, base, 2, dims, strides, box, FP8)) return false;
      for (auto [map, slots] : {std::pair<CUtensorMap*, int>{&m.box8, 8}, {&m.box32, 32},
                                {&m.box128, kTileKeys}}) {
        const cuuint32_t box3[3] = {kBoxCols, 1, (cuuint32_t)slots};
        if (!encode(map, base, 3, dims3, strides3, box3, FP8)) return false;
      }
      return true;
    };
    // with no keys no tile is ever loaded; the query buffer stands in as a valid address
    if (!pool(tk, empty ? a.q : a.k_pool) || !pool(tv, empty ? a.q : a.v_pool))
      return SEG_ATTN_ERR_CUDA;
  }
  PrefillParams p;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.tab = a.tab;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.q_heads = d.q_heads;
  p.kv_heads = d.kv_heads;
  p.group = group;
  p.qpt = d.queries_per_tile;
  p.causal = d.causal;
  p.part_o = a.part_o;
  p.part_lse = a.part_lse;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.wait_ns = g_stall_wait_ns.load();
  p.withhold_tile = g_stall_tile.load();
  p.p_delay_ns = g_order_delay_ns.load();
  p.mask_base = a.mask_base;
  p.draft_slot = a.draft_slot;
  p.v_pool = a.v_pool;
  // two-tile items first, then the single-tile items listed at the end.  A pass in
  // which some piece writes final rows runs the instantiation whose epilogue stores
  // full query tiles by TMA; a pass of partials only (every item split, or a pass
  // over shared prefixes) keeps the leaner epilogue, which measured faster there.
  const int n_single = d.num_single, n_two = d.num_work - d.num_single;
  // Drafted tokens always run the former: their passes are mostly unsplit.
  const bool any_final = TREE || d.num_parts < d.num_work;
  auto launch = [&](auto single_tag, auto tma_tag, int base, int n) {
    p.work_base = base;
    return launch_items<D, decltype(single_tag)::value, FP8, decltype(tma_tag)::value || TREE, TREE>(
        tq, to, tk, tv, p, n, stream);
  };
  using T = std::true_type;
  using F = std::false_type;
  if (n_two > 0) {
    const int rc = any_final ? launch(F{}, T{}, 0, n_two) : launch(F{}, F{}, 0, n_two);
    if (rc != SEG_ATTN_OK) return rc;
  }
  if constexpr (!TREE) {  // drafted tokens: one-tile items run both ways in one launch
    if (n_single > 0) {
      const int rc =
          any_final ? launch(T{}, T{}, n_two, n_single) : launch(T{}, F{}, n_two, n_single);
      if (rc != SEG_ATTN_OK) return rc;
    }
  }
  if (!TREE && d.num_merge > 0) {
    prefill_merge_kernel<D><<<dim3(d.num_merge, 4), 256, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  }
  return SEG_ATTN_OK;
}

}  // namespace

int launch_prefill(const PrefillLaunch& a, cudaStream_t stream) {
  auto launch = [&](auto fp8_tag, auto tree_tag) {
    constexpr bool F = decltype(fp8_tag)::value, T = decltype(tree_tag)::value;
    return a.desc->head_dim == 128 ? launch_prefill_d<128, F, T>(a, stream)
                                   : launch_prefill_d<64, F, T>(a, stream);
  };
  std::true_type yes;
  std::false_type no;
  if (a.mask_base) return a.fp8 ? launch(yes, yes) : launch(no, yes);
  return a.fp8 ? launch(yes, no) : launch(no, no);
}

namespace {

// Diagnostic: one warp waits, with the same bounded wait every kernel of this
// library uses, on an mbarrier that nothing ever arrives on.  The wait gives up
// after limit_ns and the grid records it in the device error word, as a stalled
// prefill or linear-attention kernel would.
__global__ void __launch_bounds__(32) wait_selftest_kernel(uint64_t limit_ns) {
  using namespace ptx;
  __shared__ uint64_t bar;
  __shared__ volatile int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  const bool done = mbar_wait(&bar, 0, &abort_flag, limit_ns);
  __syncwarp();
  if (threadIdx.x == 0 && (!done || abort_flag)) atomicOr(&g_device_error, 1);
}

}  // namespace

int set_order_test(int delay_ns) {
  g_order_delay_ns.store(delay_ns);
  return SEG_ATTN_OK;
}

int set_stall_test(int withhold_k_tile, int wait_us) {
  g_stall_tile.store(withhold_k_tile < 0 ? -1 : withhold_k_tile);
  g_stall_wait_ns.store((uint64_t)wait_us * 1000ull);
  return SEG_ATTN_OK;
}

int launch_wait_selftest(int wait_us, cudaStream_t stream) {
  wait_selftest_kernel<<<1, 32, 0, stream>>>((uint64_t)wait_us * 1000ull);
  return cudaGetLastError() == cudaSuccess ? SEG_ATTN_OK : SEG_ATTN_ERR_CUDA;
}

int take_device_error(int* value) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return SEG_ATTN_ERR_CUDA;
  *value = v;
  return SEG_ATTN_OK;
}

}  // namespace segattn
