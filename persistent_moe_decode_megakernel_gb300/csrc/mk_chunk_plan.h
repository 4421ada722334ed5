// mk_chunk_plan.h -- which work each block of mk_chunk_attention takes: made on the host from the
// lengths, walked by every role of a block on the device, and inspected by host tests.
//
// A UNIT is up to two tiles of query rows of one sequence (2*TT tokens); an ITEM is a unit and
// a KV head, `tiles` position tiles long; a SEGMENT is a range of an item's position tiles
// that one block runs.  Items are ordered by sequence, longest first, then from the last unit (most
// positions) to the first, then by KV head.  Two schedules:
//   whole:  blocks take whole items in alternating order (0..B-1, then B-1..0, and so on);
//   ranged: the items' position tiles, laid end to end, are cut into one contiguous range per
//           block, of equal cost; an item that a cut falls into is merged by a second kernel
//           from its blocks' partial (O, m, l), in block order.
// make_plan picks the one whose slowest block it expects to end first.
#ifndef MK_CHUNK_PLAN_H
#define MK_CHUNK_PLAN_H

#include "mk_chunk.h"

namespace mk {

constexpr int kTile = 128;           // positions of a tile, and rows of a tile
constexpr int kMaxBlocks = 152;      // one block per SM
// Position tiles that are summed in tensor memory before the sum moves into the workspace: see fold.
constexpr int kFoldTiles = 2048;

struct AttnPlan {
  static constexpr bool kSpans = false;
  int32_t n;                         // sequences with rows
  int32_t items, blocks, ranged;
  int32_t G, TT, Hkv;
  int32_t urows;                     // rows of a partial
  int32_t by_G;                      // row / G = row * by_G >> 16 for a unit's rows
  int32_t seq[kMaxSeqs];             // longest first
  int32_t units[kMaxSeqs];           // of the i-th
  int32_t item0[kMaxSeqs + 1];       // first item of the i-th
  struct { int32_t item, tile; } start[kMaxBlocks + 1];   // ranged: where each block's range begins
  int32_t cuts;                      // items that a cut falls into, and of each
  uint8_t cut_block[kMaxBlocks];     // the block that runs its beginning,
  uint8_t cut_parts[kMaxBlocks];     // and its partials: that block's and the next ones'
};

struct Segment {
  int32_t s, unit, kvh;
  int32_t tok0, ntok;                // tokens of the unit within the sequence's new ones
  int32_t pos0, len;                 // position of its first token; length of the sequence
  int32_t tile0, n, tiles;           // position tiles [tile0, tile0 + n) of the item's `tiles`
  int32_t slot;                      // partial it writes, -1: it is the whole item and writes the output
  bool two;                          // two tiles of rows (else one)
  // parts of the cache (mk_span_plan.h), where len, pos0 and tiles count places:
  int32_t entry, row0;               // its entry; first packed row
  int32_t head, gap;                 // place v is position v below `head`, v + gap from there on
  bool pair;                         // KV heads kvh and kvh + 1: n counts both heads' tiles, in turn
};

__host__ __device__ inline void item_of(const AttnPlan& pl, const ChunkSeqs& q, int item, Segment& g) {
  int lo = 0, hi = pl.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.item0[mid] <= item) lo = mid;
    else hi = mid;
  }
  g.s = pl.seq[lo];
  g.len = q.len[g.s];
  const int chunk = q.row0[g.s + 1] - q.row0[g.s], UT = 2 * pl.TT;
  const int rem = item - pl.item0[lo], back = rem / pl.Hkv;
  g.unit = pl.units[lo] - 1 - back;
  g.kvh = rem - back * pl.Hkv;
  g.tok0 = g.unit * UT;
  g.ntok = chunk - g.tok0 < UT ? chunk - g.tok0 : UT;
  g.pos0 = g.len - chunk + g.tok0;
  g.two = g.ntok > pl.TT;
  g.tiles = (g.pos0 + g.ntok - 1) / kTile + 1;
}

// Walks one block's segments.  (Whole items' partials: see mk_span_plan.h.)
struct SegmentWalk {
  int b, k, item, tile, entry;
  template <class Plan>
  __host__ __device__ SegmentWalk(const Plan& pl, int block) : b(block), k(0), item(0), tile(0), entry(0) {
    if constexpr (Plan::kSpans) entry = pl.start[b].entry;
    if (pl.ranged) {
      item = pl.start[b].item;
      tile = pl.start[b].tile;
    }
  }
  template <class Plan>
  __host__ __device__ bool next(const Plan& pl, const ChunkSeqs& q, Segment& g) {
    if (!pl.ranged) {
      const int64_t i = static_cast<int64_t>(k) * pl.blocks + (k & 1 ? pl.blocks - 1 - b : b);
      ++k;
      if (i >= pl.items) return false;   // (the last round may skip a block; no later round has items)
      look(pl, q, static_cast<int>(i), g);
      g.tile0 = 0;
      g.n = steps(pl, g, g.tiles);
      g.slot = whole_slot(pl, g);
      return true;
    }
    const int ei = pl.start[b + 1].item, et = pl.start[b + 1].tile;
    if (item > ei || (item == ei && tile >= et)) return false;
    look(pl, q, item, g);
    const int end = item == ei ? et : g.tiles;
    g.tile0 = tile;
    g.n = steps(pl, g, end - tile);
    g.slot = tile == 0 && end == g.tiles ? whole_slot(pl, g) : 2 * b + (tile == 0 ? 1 : 0);
    ++item;
    tile = 0;
    return true;
  }
  // (items rise: an entry is looked for from the last one's on)
  template <class Plan>
  __host__ __device__ void look(const Plan& pl, const ChunkSeqs& q, int i, Segment& g) {
    if constexpr (Plan::kSpans) {
      while (entry + 1 < pl.n && pl.e[entry + 1].item0 <= i) ++entry;
      item_of_entry(pl, entry, i, g);
    } else {
      item_of(pl, q, i, g);
    }
  }
  template <class Plan>
  __host__ __device__ static int steps(const Plan&, const Segment& g, int tiles) {
    if constexpr (Plan::kSpans) return g.pair ? 2 * tiles : tiles;
    else return tiles;
  }
  template <class Plan>
  __host__ __device__ static int whole_slot(const Plan& pl, const Segment& g) {
    if constexpr (Plan::kSpans) return pl.e[g.entry].part0 >= 0 ? Plan::kWholeSlot : -1;
    else return -1;
  }
};

// Floats of the workspace that a launch's blocks fold into, two streams of 128 rows each (0: no segment is so long).
template <class Plan>
size_t fold_floats(const Plan& pl, const ChunkSeqs& q, int head_dim) {
  Segment g;
  bool any = false;                  // an item is so long
  if constexpr (Plan::kSpans) {      // (a window's last unit may have three tiles fewer than the others)
    for (int i = 0; i < pl.n; ++i) {
      unit_of(pl, i, pl.e[i].units - 1, 0, g);
      any |= g.tiles + 3 > kFoldTiles;
    }
  } else if (pl.items > 0) {
    item_of(pl, q, 0, g);
    any = g.tiles > kFoldTiles;
  }
  if (any && pl.ranged) {            // and what a block has of it
    any = false;
    for (int b = 0; b < pl.blocks && !any; ++b) {
      SegmentWalk walk(pl, b);
      while (!any && walk.next(pl, q, g)) any = (g.two ? g.n : (g.n + 1) / 2) > kFoldTiles;
    }
  }
  return any ? static_cast<size_t>(pl.blocks) * 2 * kTile * (head_dim + 4) : 0;
}

// Fills the plan of the sequences that `use` marks; *floats is the size of the partials (0: none).  False: more items
// than a call takes.
bool make_plan(const mk_cache_shape& c, const ChunkSeqs& q, const bool* use, AttnPlan* pl, size_t* floats);

}  // namespace mk

#endif
