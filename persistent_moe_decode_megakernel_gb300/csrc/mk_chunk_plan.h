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

struct AttnPlan {
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

// Walks one block's segments.
struct SegmentWalk {
  int b, k, item, tile;
  __host__ __device__ SegmentWalk(const AttnPlan& pl, int block) : b(block), k(0), item(0), tile(0) {
    if (pl.ranged) {
      item = pl.start[b].item;
      tile = pl.start[b].tile;
    }
  }
  __host__ __device__ bool next(const AttnPlan& pl, const ChunkSeqs& q, Segment& g) {
    if (!pl.ranged) {
      const int64_t i = static_cast<int64_t>(k) * pl.blocks + (k & 1 ? pl.blocks - 1 - b : b);
      ++k;
      if (i >= pl.items) return false;   // (the last round may skip a block; no later round has items)
      item_of(pl, q, static_cast<int>(i), g);
      g.tile0 = 0;
      g.n = g.tiles;
      g.slot = -1;
      return true;
    }
    const int ei = pl.start[b + 1].item, et = pl.start[b + 1].tile;
    if (item > ei || (item == ei && tile >= et)) return false;
    item_of(pl, q, item, g);
    const int end = item == ei ? et : g.tiles;
    g.tile0 = tile;
    g.n = end - tile;
    g.slot = tile == 0 && end == g.tiles ? -1 : 2 * b + (tile == 0 ? 1 : 0);
    ++item;
    tile = 0;
    return true;
  }
};

// Fills the plan of the sequences that `use` marks; *floats is the size of the partials (0: none).  False: more items
// than a call takes.
bool make_plan(const mk_cache_shape& c, const ChunkSeqs& q, const bool* use, AttnPlan* pl, size_t* floats);

}  // namespace mk

#endif
