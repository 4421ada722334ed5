// mk_span_plan.h -- the schedule of attention over parts of the cache (mk_window_attention, mk_prefix_attention):
// made on the host, walked by every role of a block on the device, and inspected by host tests.
//
// An ENTRY is a run of packed rows and the positions that they go over: a sequence's rows over its own positions,
// or the rows of all sequences of a group over the positions that these share.  Its units, items, segments and
// the two schedules are those of mk_chunk_plan.h.  What differs is which positions a unit's tiles hold.  A unit's
// rows see an interval that ends with its last token and, behind a gap, the first `sinks` positions.  So its tiles
// run over PLACES: place v is position v in the head and position v + gap behind it, where head and gap are multiples
// of a copy's positions.  A window's tiles begin where its first row's does, not at a multiple of 128, and the sinks
// take the room of a copy or two instead of a tile of their own.
//
// An entry of one tile of rows (a few tokens, as in decoding) takes two KV heads at a time where their number is even: the
// block's two streams, which are even and odd position tiles of an item otherwise, are the heads then, so that short items
// are half as many and end without a join of the streams.
//
// Rows of a group have two items' worth of weights, the shared positions' and their own sequence's: such segments
// write a partial (m, l, O) each, which a second kernel joins.
#ifndef MK_SPAN_PLAN_H
#define MK_SPAN_PLAN_H

#include "mk_chunk_plan.h"

namespace mk {

constexpr int kMaxGroups = kMaxSeqs / 2;                 // groups of two sequences or more
constexpr int kMaxEntries = kMaxSeqs + kMaxGroups;
// Reaches back to position 0 from every row: no sequence is longer than 2^30, but rows that go over shared positions together
// stand behind these one after the other, up to kMaxSeqs times a unit's 2 * kTile.
constexpr int32_t kNoWindow = (1 << 30) + kMaxSeqs * 2 * kTile;

struct SpanEntry {
  int32_t seq;                       // whose block table it reads
  int32_t row0, rows;                // packed rows
  int32_t before;                    // position of its first row (shared positions: their number, so that all are before)
  int32_t from, len;                 // positions [from, len); from is a multiple of a copy's
  int32_t units, item0;
  int32_t pair;                      // 1: an item is two KV heads
  int32_t part0;                     // rows of partials before its own, -1: it writes the output
  int32_t stage0, stage_tile0, stage_head;   // q8_0 staged: its first tile in the workspace; the position tile that
                                             // follows the first stage_head ones there
};

struct SpanPlan {
  static constexpr bool kSpans = true;
  static constexpr int kWholeSlot = 2 * kMaxBlocks;      // Segment.slot of a whole item that writes a partial
  int32_t n;                         // entries: of shared positions, of sequences (those with most positions first)
  int32_t items, blocks, ranged;
  int32_t G, TT, Hkv;
  int32_t urows;                     // rows of a cut item's partial
  int32_t by_G;
  int32_t window, sinks, box;        // box: positions of a copy, a power of two
  SpanEntry e[kMaxEntries];
  struct { int32_t item, tile, entry; } start[kMaxBlocks + 1];   // (entry: of the block's first item, in ranges or not)
  int32_t cuts;                      // cut items that write the output
  uint8_t cut_block[kMaxBlocks], cut_parts[kMaxBlocks];
};

__host__ __device__ inline void unit_of(const SpanPlan& pl, int i, int unit, int kvh, Segment& g) {
  const SpanEntry& e = pl.e[i];
  const int UT = 2 * pl.TT;
  g.s = e.seq;
  g.entry = i;
  g.unit = unit;
  g.kvh = kvh;
  g.pair = e.pair != 0;
  g.tok0 = unit * UT;
  g.row0 = e.row0 + g.tok0;
  g.ntok = e.rows - g.tok0 < UT ? e.rows - g.tok0 : UT;
  g.two = g.ntok > pl.TT;
  const int pos0 = e.before + g.tok0, last = pos0 + g.ntok;
  const int end = e.len < last ? e.len : last;
  int lo = pos0 - pl.window + 1;                         // the first position in some row's window
  lo = (lo > e.from ? lo : e.from) & -pl.box;
  const int head = (pl.sinks + pl.box - 1) & -pl.box;
  g.head = lo > head ? head : 0;
  g.gap = lo > head ? lo - head : 0;
  g.pos0 = pos0 - g.gap;                                 // places from here on
  g.len = e.len - g.gap;
  g.tiles = (end - g.gap + kTile - 1) / kTile;
}

__host__ __device__ inline void item_of_entry(const SpanPlan& pl, int i, int item, Segment& g) {
  const int rem = item - pl.e[i].item0, heads = pl.Hkv >> pl.e[i].pair, back = rem / heads;
  unit_of(pl, i, pl.e[i].units - 1 - back, (rem - back * heads) << pl.e[i].pair, g);
}

// Of a decoded entry's positions those that no row sees, [first, first + n): its first unit, which reaches back furthest, has
// them between its first positions and its others.  They are not looked up.
__host__ __device__ inline void unseen_of(const SpanPlan& pl, int i, int& first, int& n) {
  Segment g;
  unit_of(pl, i, 0, 0, g);
  first = g.head;
  n = g.gap;
}

inline int entry_of_item(const SpanPlan& pl, int item) {
  int i = 0;
  while (i + 1 < pl.n && pl.e[i + 1].item0 <= item) ++i;
  return i;
}

// A call: a launch for each kind of rows that it has, and what joins them.
enum { kPageRows, kStagedRows, kFewRows, kRowKinds };
constexpr int kFewUnit = 32;         // rows of a unit of kFewRows
// Fills items and schedule of pl, a launch of that kind (all else of which is given); *floats is the size of
// the cut items' partials.  False: more items than a call takes.
bool make_plan(const mk_cache_shape& c, int kind, SpanPlan* pl, size_t* floats);

struct EntryRef {
  int8_t kind, entry;
};
struct JoinSeq {
  EntryRef own, over;                // a sequence's entry, its group's
  int32_t job0;
};
struct SpanCall {
  SpanPlan plan[kRowKinds];
  int32_t staged, stage_tiles;       // entries of plan[kStagedRows] in the order of their tiles
  int32_t tiles_entry[kMaxSeqs];
  int32_t joins, jobs;
  JoinSeq join[kMaxSeqs];
  int32_t whole_rows;
  size_t stage_bytes;                // workspace: staged tiles, then (floats) each launch's cut partials, whole ones, each one's folds
  size_t part0[kRowKinds], whole0, fold0[kRowKinds], folds[kRowKinds], floats;
  size_t bytes() const { return stage_bytes + floats * sizeof(float); }
};

// Positions of a copy, and what heads and gaps are multiples of.
inline int span_box(const mk_cache_shape& c) {
  const int box = c.page_size & -c.page_size;
  return box < kTile ? box : kTile;
}

bool plan_window(const mk_cache_shape& c, const ChunkSeqs& q, int32_t window, int32_t sinks, SpanCall* call);
bool plan_prefix(const mk_cache_shape& c, const ChunkSeqs& q, int32_t num_groups, const int32_t* group_seqs,
                 const int32_t* prefix_lens, SpanCall* call);

}  // namespace mk

#endif
