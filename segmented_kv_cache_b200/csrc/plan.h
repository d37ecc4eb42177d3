// Host planning shared by the table builders: segment lists, prefill items and
// the pieces they are cut into (defined in table.cpp).
#pragma once

#include <stdint.h>

#include <array>
#include <vector>

#include "seg_attn_internal.h"

namespace segattn {

using Row8 = std::array<int32_t, 8>;
using Row4 = std::array<int32_t, 4>;
// prefill piece: request, kv head, first query, first K tile | end K tile, partial
// slot (-1: none), flag (below), end of the request's segments | first packed query
// row, queries and keys of the request, segment holding the piece's first key | pool
// slot of the piece's first key when its first K tile lies inside that segment (-1:
// it does not), three words: zero, in a tree table the table's first mask word of the
// request (low and high half) and zero.
// Flag.  Plain tables: the piece belongs to the launch of the one-tile kernel (all pieces
// of a pass, or none).  Tree tables, which launch one kernel for all pieces: the item has
// queries in its first query tile only, and both softmax groups take that tile.
constexpr int kWorkInts = 16;
using Row16 = std::array<int32_t, kWorkInts>;

inline bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

struct Layout {
  int64_t n = 0;  // int32 elements so far
  int64_t take(int64_t count) {
    int64_t at = n;
    n += count;
    n = (n + 3) / 4 * 4;  // every array starts 16-byte aligned
    return at;
  }
};

// A request's keys as a segment list (start, len) in logical order.
struct Segs {
  std::vector<int32_t> start, len;
  int64_t keys() const {
    int64_t k = 0;
    for (int32_t l : len) k += l;
    return k;
  }
};

// Keys [from, from + count) of a segment list, as a segment list.
Segs cut(const Segs& s, int64_t from, int64_t count);

// One prefill item: (request, kv head, query tiles from q0) over `tiles` K tiles.
// `cascade` items write every piece as a partial for the shared-prefix merge;
// `single` items hold queries in their first 128-row query tile only.
struct PItem {
  int32_t r, g, q0, tiles;
  bool cascade, single;
};

struct Pieces {
  std::vector<Row16> work;      // two-tile pieces longest first, then single-tile ones
  std::vector<Row8> merge;      // split items that are not cascade items
  std::vector<int32_t> citem;   // per item: its index in `citems`, or -1
  int32_t slots = 0;            // partial-result slots
  int32_t single = 0;           // single-tile pieces (the tail of `work`)
};

// Cut items into pieces and order them (comments at the definitions).
void plan_pieces(const std::vector<PItem>& items, int max_split, std::vector<Row4>& citems,
                 Pieces& out);
void emit_pieces(const std::vector<PItem>& items, const std::vector<std::vector<int32_t>>& ends,
                 std::vector<Row4>& citems, Pieces& out);

// Fill the per-request words of each piece (comment at the definition).
void fill_request_words(std::vector<Row16>& work, const std::vector<int32_t>& q_off,
                        const std::vector<int32_t>& k_len, const std::vector<Segs>& lists,
                        const std::vector<int32_t>& seg_off);

}  // namespace segattn
