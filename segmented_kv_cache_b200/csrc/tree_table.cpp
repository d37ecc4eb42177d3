// Host side of the drafted-token attention: validator, mask words and work plan.
//
// The table is that of a prefill without a causal mask, whose work rows also say
// where the request's mask rows begin; the K tiles that reach past the cached keys
// look at them.
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <functional>
#include <limits>
#include <queue>
#include <utility>
#include <vector>

#include "plan.h"
#include "seg_attn_internal.h"
#include "seg_draft.h"

namespace {

using namespace segattn;

// Costs in tenths of the time a K tile of an item with one query tile takes (1.34 us: a
// bf16 cache's bytes at one SM's share of memory, d = 128).  A K tile of an item with two
// query tiles takes 1.9 us (its softmax).  A piece: start-up, first scores, drain and
// epilogue, 7 us measured.  A merge: its launch, and per piece the partial written and read
// back (128 rows x 512 bytes each way per query tile).  A table serves either cache, so
// E4M3 caches are cut by the same costs (there a K tile of both kinds of item is bound by
// its softmax: 1.6 and 1.9 us), and so are heads of 64.
constexpr int64_t kTileCost = 10, kTwoTileCost = 14, kPieceCost = 50;
constexpr double kMergeCost = 20.0, kMergePartCost = 0.23;
// The uncut plan is taken when it is this near the best: while memory bounds the pass,
// idle SMs cost less than the simulation says (32 trees of 16 over 8k keys: uncut 186 us,
// a plan simulated 4 % shorter 201; one measurement, with every K tile costed alike).
constexpr double kUncutSlack = 1.08;

// Where to cut the items along their keys: the cuts whose simulated schedule (pieces
// longest first, each to the least loaded SM) plus merge is the shortest, among
//   - every item in f equal pieces, f up to what gives each SM a few pieces;
//   - whole waves of uncut items, and the items of the last, partly filled wave in f
//     equal pieces;
//   - the items end to end, cut wherever an SM's equal share of all K tiles ends.
// `one_tile[i]`: item i has queries in its first query tile only.
std::vector<std::vector<int32_t>> plan_cuts(const std::vector<PItem>& items,
                                            const std::vector<char>& one_tile) {
  const size_t n = items.size();
  using Cuts = std::vector<std::vector<int32_t>>;
  auto equal = [&](size_t i, int64_t f, std::vector<int32_t>& ends) {
    const int64_t t = items[i].tiles, p = std::max<int64_t>(1, std::min(f, t));
    for (int64_t j = 1; j <= p; ++j) ends.push_back((int32_t)(t * j / p));
  };
  auto tile_cost = [&](size_t i) { return one_tile[i] ? kTileCost : kTwoTileCost; };
  std::vector<Cuts> cands;
  const int64_t most = std::min<int64_t>(
      2 * kSmCount, std::max<int64_t>(4, 2 * kSmCount / std::max<int64_t>(1, (int64_t)n)));
  for (int64_t f = 1; f <= most; ++f) {
    Cuts c(n);
    for (size_t i = 0; i < n; ++i) equal(i, f, c[i]);
    cands.push_back(std::move(c));
  }
  std::vector<size_t> order(n);  // longest first
  for (size_t i = 0; i < n; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(),
                   [&](size_t a, size_t b) {
                     return items[a].tiles * tile_cost(a) > items[b].tiles * tile_cost(b);
                   });
  const size_t whole = n / kSmCount * kSmCount;
  if (whole > 0 && whole < n)
    for (int64_t f = 2; f <= 8; ++f) {
      Cuts c(n);
      for (size_t k = 0; k < n; ++k) equal(order[k], k < whole ? 1 : f, c[order[k]]);
      cands.push_back(std::move(c));
    }
  int64_t total = 0;
  for (size_t i = 0; i < n; ++i) total += items[i].tiles * tile_cost(i);
  if (total >= kSmCount * kTwoTileCost) {
    // a cut that would leave fewer than kShort tiles on one side is moved to the item's end
    constexpr int64_t kShort = 4;
    Cuts c(n);
    int64_t at = 0;  // cost before item k, longest first
    for (size_t k = 0; k < n; ++k) {
      const int64_t t = items[order[k]].tiles, w = tile_cost(order[k]);
      int64_t last = 0;
      for (int64_t s = at * kSmCount / total + 1; s <= kSmCount; ++s) {
        const int64_t cut = (s * total / kSmCount - at) / w;
        if (cut >= t) break;
        if (cut - last < kShort || t - cut < kShort) continue;
        c[order[k]].push_back((int32_t)cut);
        last = cut;
      }
      c[order[k]].push_back((int32_t)t);
      at += t * w;
    }
    cands.push_back(std::move(c));
  }
  std::vector<double> all(cands.size());
  std::vector<int64_t> cost, parts(cands.size(), 0);
  for (size_t k = 0; k < cands.size(); ++k) {
    cost.clear();
    for (size_t i = 0; i < n; ++i) {
      const std::vector<int32_t>& ends = cands[k][i];
      int32_t from = 0;
      for (int32_t e : ends) {
        cost.push_back((e - from) * tile_cost(i) + kPieceCost);
        from = e;
      }
      if (ends.size() > 1) parts[k] += (int64_t)ends.size() * (one_tile[i] ? 1 : 2);
    }
    std::sort(cost.begin(), cost.end(), std::greater<int64_t>());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> sm;
    for (int i = 0; i < kSmCount; ++i) sm.push(0);
    int64_t span = 0;
    for (int64_t c : cost) {
      const int64_t t = sm.top() + c;
      sm.pop();
      sm.push(t);
      span = std::max(span, t);
    }
    all[k] = (double)span +
             (parts[k] ? kMergeCost + kMergePartCost * (double)parts[k] : 0.0);
  }
  size_t pick = std::min_element(all.begin(), all.end()) - all.begin();
  if (all[0] <= kUncutSlack * all[pick]) pick = 0;
  return std::move(cands[pick]);
}

int build(int batch, const int32_t* draft_lens, const int32_t* parents, const uint8_t* mask,
          const int32_t* seg_counts, const int32_t* seg_starts, const int32_t* seg_lens,
          int64_t num_slots, int q_heads, int kv_heads, int head_dim, void* host_out,
          size_t host_out_bytes, seg_attn_tree_desc* desc) {
  if (batch < 0 || num_slots < 0 || (parents && mask)) return SEG_ATTN_ERR_INVALID_ARG;
  if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0) return SEG_ATTN_ERR_INVALID_ARG;
  if (batch > 0 && (!seg_counts || !draft_lens)) return SEG_ATTN_ERR_INVALID_ARG;
  const int group = q_heads / kv_heads;
  if (head_dim != 64 && head_dim != 128) return SEG_ATTN_ERR_UNSUPPORTED;
  if (!is_pow2(group) || group > kTileRows) return SEG_ATTN_ERR_UNSUPPORTED;
  const int64_t kI32Max = std::numeric_limits<int32_t>::max();
  // the K/V gather addresses pool rows (slot * kv_heads + head) with int32
  if (num_slots > kI32Max / kv_heads) return SEG_ATTN_ERR_UNSUPPORTED;
  int64_t nseg_in = 0;
  for (int r = 0; r < batch; ++r) {
    if (seg_counts[r] < 0) return SEG_ATTN_ERR_INVALID_ARG;
    nseg_in += seg_counts[r];
  }
  if (nseg_in > kI32Max) return SEG_ATTN_ERR_UNSUPPORTED;
  if (nseg_in > 0 && (!seg_starts || !seg_lens)) return SEG_ATTN_ERR_INVALID_ARG;

  std::vector<int32_t> q_off(batch + 1, 0), keys(batch), draft_slot;
  std::vector<Segs> own(batch);
  std::vector<uint32_t> words;            // mask words, rows back to back
  std::vector<int64_t> mask_at(batch);    // first word of each request
  int64_t total_q = 0, total_k = 0, seg0 = 0, mask0 = 0, nseg = 0;
  int32_t max_draft = 0;
  std::vector<std::pair<int64_t, int64_t>> runs;
  for (int r = 0; r < batch; ++r) {
    Segs all;
    int64_t k = 0;
    runs.clear();
    for (int s = 0; s < seg_counts[r]; ++s) {
      const int64_t st = seg_starts[seg0 + s], ln = seg_lens[seg0 + s];
      if (ln < 0) return SEG_ATTN_ERR_INVALID_ARG;
      if (st < 0 || st + ln > num_slots) return SEG_ATTN_ERR_SEGMENT_OOB;
      k += ln;
      if (ln > 0) runs.emplace_back(st, ln);
      all.start.push_back((int32_t)st);
      all.len.push_back((int32_t)ln);
    }
    seg0 += seg_counts[r];
    std::sort(runs.begin(), runs.end());
    for (size_t i = 1; i < runs.size(); ++i)
      if (runs[i].first < runs[i - 1].first + runs[i - 1].second)
        return SEG_ATTN_ERR_SEGMENT_OVERLAP;
    if (k > kI32Max) return SEG_ATTN_ERR_UNSUPPORTED;
    const int32_t t = draft_lens[r];
    if (t < 0) return SEG_ATTN_ERR_INVALID_ARG;
    if (t > SEG_ATTN_TREE_MAX_DRAFT) return SEG_ATTN_ERR_UNSUPPORTED;
    if (t > k) return SEG_ATTN_ERR_QLEN_GT_KLEN;
    keys[r] = (int32_t)k;
    own[r] = cut(all, 0, k);  // without empty segments
    nseg += (int64_t)own[r].len.size();
    const Segs drafts = cut(all, k - t, t);
    for (size_t i = 0; i < drafts.len.size(); ++i)
      for (int32_t j = 0; j < drafts.len[i]; ++j) draft_slot.push_back(drafts.start[i] + j);
    // mask rows
    const int32_t nw = (t + 31) / 32;
    mask_at[r] = (int64_t)words.size();
    words.resize(words.size() + (size_t)t * nw, 0u);
    uint32_t* rows = words.data() + mask_at[r];
    for (int32_t i = 0; i < t; ++i) {
      uint32_t* row = rows + (size_t)i * nw;
      if (mask) {
        const uint8_t* m = mask + mask0 + (int64_t)i * t;
        for (int32_t j = 0; j < t; ++j)
          if (m[j]) row[j >> 5] |= 1u << (j & 31);
        continue;
      }
      const int32_t p = parents ? parents[total_q + i] : i - 1;
      if (p < -1 || p >= i) return SEG_ATTN_ERR_INVALID_ARG;
      if (p >= 0)
        for (int32_t w = 0; w < nw; ++w) row[w] = rows[(size_t)p * nw + w];
      row[i >> 5] |= 1u << (i & 31);
    }
    mask0 += (int64_t)t * t;
    total_q += t;
    total_k += k;
    if (total_q > kI32Max) return SEG_ATTN_ERR_UNSUPPORTED;
    q_off[r + 1] = (int32_t)total_q;
    max_draft = std::max(max_draft, t);
  }

  // ---- work plan
  const int32_t qpt = kTileRows / group;
  const int32_t span = qpt * kTilesPerItem;
  std::vector<PItem> items;
  std::vector<char> one_tile;  // both softmax groups take the item's one query tile
  int32_t max_k_tiles = 0;
  for (int r = 0; r < batch; ++r) {
    const int32_t t = q_off[r + 1] - q_off[r];
    const int32_t tiles = (int32_t)(((int64_t)keys[r] + kTileKeys - 1) / kTileKeys);
    max_k_tiles = std::max(max_k_tiles, tiles);
    for (int32_t q0 = 0; q0 < t; q0 += span)
      for (int g = 0; g < kv_heads; ++g) {
        items.push_back({r, g, q0, tiles, false, false});
        one_tile.push_back(t - q0 <= qpt);
      }
  }
  std::vector<Row4> no_citems;
  Pieces pieces;
  emit_pieces(items, plan_cuts(items, one_tile), no_citems, pieces);
  if (pieces.work.size() > (size_t)kI32Max) return SEG_ATTN_ERR_UNSUPPORTED;

  // ---- layout
  Layout lay;
  seg_attn_table_desc& p = desc->pass;
  p.off_q_offsets = lay.take(batch + 1);
  p.off_k_lens = lay.take(batch);
  p.off_seg_offsets = lay.take(batch + 1);
  p.off_seg_start = lay.take(nseg);
  p.off_seg_kstart = lay.take(nseg);
  p.off_seg_len = lay.take(nseg);
  p.off_work = lay.take(kWorkInts * (int64_t)pieces.work.size());
  p.off_merge = lay.take(8 * (int64_t)pieces.merge.size());
  desc->off_mask = lay.take((int64_t)words.size());
  desc->off_draft_slot = lay.take(total_q);

  p.magic = SEG_ATTN_TREE_MAGIC;  // not a table the plain calls take
  p.version = SEG_ATTN_TABLE_VERSION;
  p.mode = SEG_ATTN_MODE_PREFILL;
  p.batch = batch;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.head_dim = head_dim;
  p.num_slots = num_slots;
  p.total_q = total_q;
  p.total_k = total_k;
  p.num_segments = (int32_t)nseg;
  p.num_work = (int32_t)pieces.work.size();
  p.queries_per_tile = qpt;
  p.max_k_tiles = max_k_tiles;
  p.num_merge = (int32_t)pieces.merge.size();
  p.num_parts = pieces.slots;
  desc->magic = SEG_ATTN_TREE_MAGIC;
  desc->version = SEG_ATTN_TREE_VERSION;
  desc->batch = batch;
  desc->max_draft = max_draft;
  desc->table_bytes = (uint64_t)lay.n * sizeof(int32_t);
  desc->workspace_bytes = workspace_layout(p, false).total;
  p.table_bytes = desc->table_bytes;
  p.workspace_bytes = desc->workspace_bytes;

  if (!host_out) return SEG_ATTN_OK;  // size query
  if (host_out_bytes < desc->table_bytes) return SEG_ATTN_ERR_BUFFER_TOO_SMALL;
  if ((reinterpret_cast<uintptr_t>(host_out) & 15) != 0) return SEG_ATTN_ERR_INVALID_ARG;

  int32_t* t = static_cast<int32_t*>(host_out);
  memset(t, 0, desc->table_bytes);
  memcpy(t + p.off_q_offsets, q_off.data(), q_off.size() * sizeof(int32_t));
  std::vector<int32_t> seg_off(batch + 1, 0);
  int32_t s0 = 0;
  for (int r = 0; r < batch; ++r) {
    t[p.off_k_lens + r] = keys[r];
    int32_t logical = 0;
    for (size_t s = 0; s < own[r].len.size(); ++s, ++s0) {
      t[p.off_seg_start + s0] = own[r].start[s];
      t[p.off_seg_kstart + s0] = logical;
      t[p.off_seg_len + s0] = own[r].len[s];
      logical += own[r].len[s];
    }
    seg_off[r + 1] = s0;
    t[p.off_seg_offsets + r + 1] = s0;
  }
  fill_request_words(pieces.work, q_off, keys, own, seg_off);
  for (size_t i = 0; i < pieces.work.size(); ++i) {
    const int64_t at = desc->off_mask + mask_at[pieces.work[i][0]];
    // both softmax groups take the one query tile of such an item.  Set here, after
    // emit_pieces has ordered the pieces longest first: one launch runs both kinds.
    pieces.work[i][6] = q_off[pieces.work[i][0] + 1] - q_off[pieces.work[i][0]] - pieces.work[i][2] <= qpt;
    pieces.work[i][13] = (int32_t)(uint32_t)(at & 0xffffffff);
    pieces.work[i][14] = (int32_t)(at >> 32);
    memcpy(t + p.off_work + kWorkInts * i, pieces.work[i].data(), kWorkInts * sizeof(int32_t));
  }
  for (size_t i = 0; i < pieces.merge.size(); ++i)
    memcpy(t + p.off_merge + 8 * i, pieces.merge[i].data(), 8 * sizeof(int32_t));
  if (!words.empty()) memcpy(t + desc->off_mask, words.data(), words.size() * sizeof(uint32_t));
  if (!draft_slot.empty())
    memcpy(t + desc->off_draft_slot, draft_slot.data(), draft_slot.size() * sizeof(int32_t));
  return SEG_ATTN_OK;
}

}  // namespace

extern "C" int seg_attn_build_tree_table(int batch, const int32_t* draft_lens,
                                         const int32_t* parents, const uint8_t* mask,
                                         const int32_t* seg_counts, const int32_t* seg_starts,
                                         const int32_t* seg_lens, int64_t num_slots, int q_heads,
                                         int kv_heads, int head_dim, void* host_out,
                                         size_t host_out_bytes, seg_attn_tree_desc* desc) {
  if (!desc) return SEG_ATTN_ERR_INVALID_ARG;
  memset(desc, 0, sizeof(*desc));
  int rc;
  try {
    rc = build(batch, draft_lens, parents, mask, seg_counts, seg_starts, seg_lens, num_slots,
               q_heads, kv_heads, head_dim, host_out, host_out_bytes, desc);
  } catch (...) {  // host memory: no exception leaves a C entry
    rc = SEG_ATTN_ERR_UNSUPPORTED;
  }
  // a failed build leaves nothing a compute call would accept; a too small buffer
  // leaves the needed size
  if (rc != SEG_ATTN_OK) desc->magic = 0;
  return rc;
}

extern "C" size_t seg_attn_tree_workspace_size(const seg_attn_tree_desc* desc) {
  if (!desc || desc->magic != SEG_ATTN_TREE_MAGIC) return 0;
  return (size_t)desc->workspace_bytes;
}
