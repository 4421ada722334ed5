// mk_span_plan.cpp -- the schedules of mk_window_attention and mk_prefix_attention (see mk_span_plan.h).  Host only.

#include "mk_span_plan.h"

#include <algorithm>

namespace mk {

namespace {

// Costs in tenths of a microsecond, from timelines of a block's segments: a position tile, and what a segment adds to
// its tiles (the first scores and weights, the epilogue), for segments of one tile of rows, of two, and of one of two KV
// heads (both heads' tiles).  Of q8_0 the tiles' are what decoding takes.
enum { kOneTile, kTwoTiles, kTwoHeads };
struct Costs {
  int tile[3], segment[3];
};
constexpr Costs kCosts[kRowKinds] = {{{9, 16, 18}, {38, 42, 20}}, {{9, 16, 0}, {38, 42, 0}}, {{13, 0, 0}, {45, 0, 0}}};
constexpr Costs kQ8Costs = {{16, 20, 32}, {40, 32, 40}};
const Costs& costs(const mk_cache_shape& c, int kind) {
  return kind == kPageRows && (c.flags & MK_FLAG_KV_Q8) ? kQ8Costs : kCosts[kind];
}
// What cut items cost besides: the second kernel, and the bytes of partials that it and the first one move in a tenth.
constexpr int64_t kJoinCost = 45, kJoinBytes = 250000;
// Measured below: calls of 32 / 4 heads of 128 and pages of 64, over bf16 unless said, each after a pass over 512 MB, less
// that pass.
//
// What going over shared positions together costs besides: that, and the smaller pieces.  (8 sequences of 5 rows behind 8192
// positions, 7.7 us less work together: 23 us apart, 34 together; 32 tokens behind 2048, 11.3 less: 23 and 25, over q8_0 29
// and 28; 64 behind 1024: 26 and 25; 8 behind 8192: 22 and 18; 16 behind 8192, 22.6 less: 33 and 24.)  A run has to save kRunCost
// by itself.  (16 groups of 4 tokens behind 4096: 82 us apart, 44 together, and apart if a run had to save 4 us; 20 groups
// of 3 behind 2048, which this leaves apart: 40, together 38; 32 groups of 2: alike either way.)
constexpr int64_t kShareCost = 95, kRunCost = 10;
constexpr int kLeastSegment = 20;            // of these costs.  (From 1 to 60 alike; 120: one token through 4096 12.8 us for 11.7,
                                             // 64 tokens through 4096 99 for 103.)
constexpr int kMostTries = 24;
// Position tiles a block is worth.  (One token through 8192: 14.0 us with 1, 13.3 with 3, 12.8 with 5, 15.8 with 8; through
// 1024 10.4, 10.7, 13.4 and 13.2.  Over q8_0 2 would be better: one token through 4096 18.9 us, 20.5 with 3, 26.1 with 8.)
constexpr int kMinRange = 3;
constexpr int kMaxRuns = 4096;               // units beyond which whole items are even enough

// Launches are of one kind of operand each (SpanCall); a sequence's rows take
//   kFewRows  over q8_0, where its units have at most 32 rows of a KV head,
//   kStagedRows  over q8_0, where decoding their positions once, into the workspace, is less work than every unit's
//             block doing it: that costs a block 0.8 us a tile more (over all blocks), staging a launch, 5 us, and its
//             bytes, 0.025 us a tile and KV head.  (1024 rows of 16384 through 2048: 44 us, staged 43; 4096 of 8192
//             through 512: 74 and 64; 512 through 4096: 64 and 55.  Left by this rule: 512 through 256, 16 and 21; 2048
//             through 512, 40 and 39.)  kStageBytes of decoded positions at most in a call;
//   kPageRows  else.
constexpr size_t kStageBytes = size_t(1) << 30;
// Position tiles a block from which on items are of two KV heads.  (64 tokens through 128: 19.2 us with a head an item, 14.6
// with two; through 1024: 39 and 37; q8_0, 64 sequences of 5 rows through 1024: 42 and 35; 16 / 4 heads of 64, 64 tokens
// through 2048: 40 and 36: these have more items than blocks.  By their tiles alone: q8_0, 20 sequences of 5 rows through 2048,
// 36 and 34; but 71 and 74 through 8000 (over q8_0 69 and 71), 38 through 1000, an item a block, 25 and 28 (over q8_0 23.5 and
// 36), and one token through 32768 22.7 and 26.1.  So this half of the rule loses more often than it gains.)
constexpr int kPairTiles = 4;
// Position tiles a block of few rows up to which they go with another launch.  (A token of each of 63 sequences and a chunk
// of 40 through 1024: 68 us in launches of their own, 36 together; through 2048 92 and 57; through 4096, beyond: 119 and 118.)
constexpr int kGatherTiles = 40;

struct Builder {
  const mk_cache_shape& c;
  SpanCall* call;
  int G, UT;
  Builder(const mk_cache_shape& c, SpanCall* call) : c(c), call(call), G(c.num_q_heads / c.num_kv_heads), UT(2 * (kTile / G)) {}

  // adds an entry to the launch that suits it; returns where it is
  EntryRef add(SpanEntry e) {
    int kind = kPageRows;
    e.units = (e.rows + UT - 1) / UT;
    e.pair = e.stage0 = e.stage_tile0 = e.stage_head = 0;
    if (c.flags & MK_FLAG_KV_Q8) {
      if (std::min(e.rows, UT) * G <= kFewUnit) kind = kFewRows;
      else if (stage(&e)) kind = kStagedRows;
    }
    SpanPlan& pl = call->plan[kind];
    EntryRef at = {static_cast<int8_t>(kind), static_cast<int8_t>(pl.n)};
    if (kind == kStagedRows) call->tiles_entry[call->staged++] = at.entry;
    pl.e[pl.n++] = e;
    return at;
  }

  void fill(SpanPlan* pl) {
    pl->Hkv = c.num_kv_heads;
    pl->G = G;
    pl->TT = kTile / G;
    pl->by_G = 65536 / G + 1;   // exact below 2^9 rows
  }

  bool stage(SpanEntry* e) {
    SpanPlan probe;
    fill(&probe);
    probe.window = call->plan[0].window;
    probe.sinks = call->plan[0].sinks;
    probe.box = call->plan[0].box;
    probe.e[0] = *e;
    Segment g;
    unit_of(probe, 0, 0, 0, g);
    const int head = (g.head + kTile - 1) / kTile;       // (the first unit reaches back furthest)
    e->stage_tile0 = (g.head + g.gap) / kTile;
    if (g.gap == 0) e->stage_tile0 = 0;
    e->stage_head = std::min(head, e->stage_tile0);
    const int own = e->stage_head + (e->len + kTile - 1) / kTile - e->stage_tile0;
    int64_t times = 0;
    for (int u = 0; u < e->units; ++u) {
      unit_of(probe, 0, u, 0, g);
      times += g.tiles;
    }
    const size_t bytes = static_cast<size_t>(own) * 2 * c.num_kv_heads * kTile * c.head_dim * 2;
    if (times * c.num_kv_heads * 8 / kMaxBlocks <= 50 + static_cast<int64_t>(own) * c.num_kv_heads / 4 ||
        call->stage_bytes + bytes > kStageBytes)
      return false;
    e->stage0 = call->stage_tiles;
    call->stage_tiles += own;
    call->stage_bytes += bytes;
    return true;
  }

  // Few rows go with the launch that there is anyway, where the time that theirs saves them (about a quarter of a
  // microsecond a position tile) is less than what another launch takes.
  void gather() {
    SpanPlan &few = call->plan[kFewRows], &pages = call->plan[kPageRows];
    if (few.n == 0 || pages.n == 0) return;
    fill(&few);
    int64_t tiles = 0;
    Segment g;
    for (int i = 0; i < few.n; ++i) {
      unit_of(few, i, 0, 0, g);
      tiles += static_cast<int64_t>(few.e[i].units) * c.num_kv_heads * g.tiles;
    }
    if (tiles > kGatherTiles * kMaxBlocks) return;
    int moved[kMaxEntries];
    for (int i = 0; i < few.n; ++i) {
      pages.e[pages.n] = few.e[i];
      moved[i] = pages.n++;
    }
    few.n = 0;
    for (int k = 0; k < call->joins; ++k)
      for (EntryRef* r : {&call->join[k].own, &call->join[k].over})
        if (r->kind == kFewRows) *r = {kPageRows, static_cast<int8_t>(moved[r->entry])};
  }

  bool finish(const ChunkSeqs& q) {
    gather();
    size_t at = 0;
    // Two KV heads an item, where there are more items than blocks without that, or kPairTiles position tiles a block.
    // (Few rows over q8_0 stand in all lanes of a block's, so that both streams are one head's.)
    SpanPlan& pages = call->plan[kPageRows];
    fill(&pages);
    int64_t items = 0, tiles = 0;
    Segment g;
    for (int i = 0; i < pages.n; ++i) {
      unit_of(pages, i, pages.e[i].units - 1, 0, g);     // (its longest)
      items += static_cast<int64_t>(pages.e[i].units) * c.num_kv_heads;
      tiles += static_cast<int64_t>(pages.e[i].units) * c.num_kv_heads * g.tiles;
    }
    const bool pair = c.num_kv_heads % 2 == 0 && (items > kMaxBlocks || tiles > kPairTiles * kMaxBlocks);
    for (int i = 0; i < pages.n; ++i) pages.e[i].pair = pair && pages.e[i].rows <= kTile / G;
    for (int k = 0; k < kRowKinds; ++k) {
      SpanPlan& pl = call->plan[k];
      fill(&pl);
      size_t floats = 0;
      if (!make_plan(c, k, &pl, &floats)) return false;
      call->part0[k] = at;
      at += floats;
    }
    call->whole0 = at;
    at += static_cast<size_t>(call->whole_rows) * c.num_q_heads * (c.head_dim + 4);
    for (int k = 0; k < kRowKinds; ++k) {
      call->fold0[k] = at;
      at += call->folds[k] = fold_floats(call->plan[k], q, c.head_dim);
    }
    call->floats = at;
    return true;
  }
};

void reset(const mk_cache_shape& c, int window, int sinks, SpanCall* call) {
  for (SpanPlan& pl : call->plan) {
    pl.n = 0;
    pl.window = window;
    pl.sinks = sinks;
    pl.box = span_box(c);
  }
  call->staged = call->stage_tiles = call->joins = call->jobs = 0;
  call->stage_bytes = 0;
  call->whole_rows = 0;
}

// The sequences with rows, the longest first.
int by_length(const ChunkSeqs& q, int* order) {
  int n = 0;
  for (int s = 0; s < q.n; ++s)
    if (q.row0[s + 1] > q.row0[s]) order[n++] = s;
  std::sort(order, order + n, [&](int a, int b) { return q.len[a] != q.len[b] ? q.len[a] > q.len[b] : a < b; });
  return n;
}

SpanEntry entry_of(const ChunkSeqs& q, int s) {
  SpanEntry e = {};
  e.seq = s;
  e.row0 = q.row0[s];
  e.rows = q.row0[s + 1] - q.row0[s];
  e.before = q.len[s] - e.rows;
  e.len = q.len[s];
  e.part0 = -1;
  return e;
}

}  // namespace

bool make_plan(const mk_cache_shape& c, int kind, SpanPlan* pl, size_t* floats) {
  pl->blocks = pl->ranged = pl->cuts = 0;
  *floats = 0;
  const Costs& cost = costs(c, kind);
  // runs of items that are alike: a unit's KV heads, and those of units behind it
  struct Run {
    int32_t tiles, items;
    int16_t type, rows;
  };
  Run run[kMaxRuns];
  int runs = 0, most = 0;
  int64_t items = 0, tiles = 0, work = 0;
  for (int i = 0; i < pl->n; ++i) {
    SpanEntry& e = pl->e[i];
    most = std::max(most, std::min(e.rows, 2 * pl->TT) << e.pair);
    e.item0 = static_cast<int32_t>(items);
    const int heads = pl->Hkv >> e.pair;
    items += static_cast<int64_t>(e.units) * heads;
    if (items >= (int64_t(1) << 31)) return false;
    if (e.units > kMaxRuns - runs) {
      runs = kMaxRuns + 1;
      continue;
    }
    Segment g;
    for (int u = e.units - 1; u >= 0; --u) {
      unit_of(*pl, i, u, 0, g);
      const int type = g.two ? kTwoTiles : g.pair ? kTwoHeads : kOneTile;
      const int16_t rows = static_cast<int16_t>(g.ntok * pl->G << e.pair);
      Run* last = run + runs - 1;
      if (runs > 0 && last->tiles == g.tiles && last->type == type && last->rows == rows) last->items += heads;
      else run[runs++] = {g.tiles, heads, static_cast<int16_t>(type), rows};
      tiles += static_cast<int64_t>(g.tiles) * heads;
      work += (static_cast<int64_t>(g.tiles) * cost.tile[type] + cost.segment[type]) * heads;
    }
  }
  pl->urows = most * pl->G;
  pl->items = static_cast<int32_t>(items);
  pl->blocks = std::min<int32_t>(pl->items, kMaxBlocks);
  if (items > 0 && runs <= kMaxRuns) {
    // the slowest block of whole items
    int64_t load[kMaxBlocks] = {};
    for (int i = 0, b = 0, step = 1; i < runs; ++i) {
      const int64_t x = static_cast<int64_t>(run[i].tiles) * cost.tile[run[i].type] + cost.segment[run[i].type];
      for (int k = 0; k < run[i].items; ++k) {
        load[b] += x;
        b += step;                           // 0..B-1, then B-1..0
        if (b == pl->blocks || b < 0) {
          step = -step;
          b += step;
        }
      }
    }
    const int64_t whole = *std::max_element(load, load + pl->blocks);
    const int nb = static_cast<int>(std::min<int64_t>(kMaxBlocks, (tiles + kMinRange - 1) / kMinRange));
    // Ranges: each block takes segments up to `limit`.  Whether that is enough for all items.
    int64_t partials = 0;
    auto cut = [&](int32_t limit) {
      int b = 0, item = 0;
      int32_t left = limit;
      partials = 0;
      pl->start[0].item = pl->start[0].tile = 0;
      for (int i = 0; i < runs; ++i) {
        const int32_t per = cost.tile[run[i].type], own = cost.segment[run[i].type], all = run[i].tiles;
        const int64_t one = own + static_cast<int64_t>(per) * all;
        for (int k = 0, at = 0; k < run[i].items;) {
          if (at == 0 && left >= one) {                    // whole items
            const int fit = std::min<int32_t>(run[i].items - k, left / static_cast<int32_t>(one));
            k += fit;
            item += fit;
            left -= fit * static_cast<int32_t>(one);
            continue;
          }
          int32_t n = left < own ? 0 : (left - own) / per;
          if (n > 0 && n + 1 >= all - at) n = all - at;    // (a last tile is not worth a segment,
          if (n == 0 || (n == 1 && n < all - at && left < limit)) {   // nor is a first one)
            if (++b >= nb || (n == 0 && limit < own + per)) return false;
            left = limit;
            pl->start[b].item = item;
            pl->start[b].tile = at;
            continue;
          }
          if (n < all) partials += run[i].rows;
          at += n;
          left -= own + n * per;
          if (at == all) {
            at = 0;
            ++k;
            ++item;
          }
        }
      }
      pl->blocks = b + 1;
      pl->start[b + 1].item = pl->items;
      pl->start[b + 1].tile = 0;
      return true;
    };
    // Every block but the first begins inside an item, about: a segment more than its share of the work.  From three quarters
    // of that (a quarter to all of it: within 1 % over bf16; half as much again: 64 tokens behind 32768 54 us for 52) the
    // limit rises until it is enough.
    const int64_t share = work / nb;
    int64_t more = 0;
    for (int i = 0; i < runs; ++i)
      more += static_cast<int64_t>(run[i].tiles) * cost.tile[run[i].type] * run[i].items / std::max<int64_t>(share, 1) *
              cost.segment[run[i].type];
    more = more / nb * 3 / 4;
    int64_t limit = share + std::max<int64_t>(more, kLeastSegment / 2);
    if (limit + kJoinCost < whole && limit < (int64_t(1) << 30)) {
      const int64_t step = std::max<int64_t>(limit / 64, 4);
      bool enough = false;
      for (int i = 0; i < kMostTries && !(enough = cut(static_cast<int32_t>(limit))); ++i) limit += step;
      if (enough && limit + kJoinCost + partials * (c.head_dim + 4) * 8 / kJoinBytes < whole) {
        pl->ranged = 1;
        *floats = static_cast<size_t>(2) * pl->blocks * pl->urows * (c.head_dim + 4);
      } else {
        pl->blocks = std::min<int32_t>(pl->items, kMaxBlocks);
      }
    }
  }
  for (int b = 0, i = 0; b < pl->blocks; ++b) {
    const int item = pl->ranged ? pl->start[b].item : b;
    while (i + 1 < pl->n && pl->e[i + 1].item0 <= item) ++i;
    pl->start[b].entry = i;
    // an item that is cut and writes the output: by its first block, with the blocks whose ranges begin inside it
    if (!pl->ranged || pl->start[b + 1].tile == 0) continue;
    const int last = pl->start[b + 1].item;
    if (pl->start[b].item == last && pl->start[b].tile > 0) continue;
    int e = i, n = 2;
    while (e + 1 < pl->n && pl->e[e + 1].item0 <= last) ++e;
    if (pl->e[e].part0 >= 0) continue;
    while (b + n <= pl->blocks && pl->start[b + n].item == last) ++n;
    pl->cut_block[pl->cuts] = static_cast<uint8_t>(b);
    pl->cut_parts[pl->cuts++] = static_cast<uint8_t>(n);
  }
  return true;
}

bool plan_window(const mk_cache_shape& c, const ChunkSeqs& q, int32_t window, int32_t sinks, SpanCall* call) {
  reset(c, std::min(window, kNoWindow), std::min(sinks, kNoWindow), call);
  Builder build(c, call);
  int order[kMaxSeqs];
  const int n = by_length(q, order);
  for (int i = 0; i < n; ++i) build.add(entry_of(q, order[i]));
  return build.finish(q);
}

bool plan_prefix(const mk_cache_shape& c, const ChunkSeqs& q, int32_t num_groups, const int32_t* group_seqs,
                 const int32_t* prefix_lens, SpanCall* call) {
  reset(c, kNoWindow, 0, call);
  Builder build(c, call);
  const int UT = build.UT;
  // Runs of a group's sequences whose rows do not fill a unit of their own (with others', they share one), between those
  // that do.  A run's rows may go over the shared positions together where that saves blocks time (over all of them), and
  // the runs of which that holds do so if they save more than that costs.
  struct { int32_t first, end, positions; } run[kMaxSeqs];
  int runs = 0;
  int64_t total = 0;
  int32_t common[kMaxSeqs];                              // whole pages that a sequence's run goes over together, or 0
  EntryRef over[kMaxSeqs];
  for (int i = 0, s0 = 0; i < num_groups; s0 += group_seqs[i++]) {
    const int positions = prefix_lens[i] / c.page_size * c.page_size, tiles = (positions + kTile - 1) / kTile;
    const Costs& x = costs(c, kPageRows);
    auto cost = [&](int rows, int item) {                // (a unit of more than half its rows has two tiles)
      const int full = rows / UT + (rows % UT > UT / 2), rest = rows % UT > 0 && rows % UT <= UT / 2;
      return static_cast<int64_t>(full) * (tiles * x.tile[kTwoTiles] + item * x.segment[kTwoTiles]) +
             rest * (tiles * x.tile[kOneTile] + item * x.segment[kOneTile]);
    };
    for (int s = s0, end = s0 + group_seqs[i]; s < end;) {
      const int first = s;
      int with = 0;
      int64_t apart = 0;
      for (; s < end && q.row0[s + 1] - q.row0[s] < UT; ++s) {
        apart += cost(q.row0[s + 1] - q.row0[s], 0);
        with += q.row0[s + 1] > q.row0[s];
        common[s] = 0;
      }
      const int rows = q.row0[s] - q.row0[first];
      if (with > 1 && tiles > 0) {
        const int64_t saved = (apart - cost(rows, 1)) * c.num_kv_heads / kMaxBlocks;
        const int64_t bytes = static_cast<int64_t>(rows) * c.num_q_heads * (c.head_dim + 4) * 8;
        if (saved > kRunCost + bytes / kJoinBytes) {
          run[runs++] = {first, s, positions};
          total += saved - bytes / kJoinBytes;
        }
      }
      if (s < end && s == first) common[s++] = 0;         // fills units of its own
    }
  }
  for (int i = 0; i < runs && total > kShareCost; ++i) {
    SpanEntry e = {};
    e.seq = run[i].first;                                 // (the first with rows: another's table is not read)
    while (q.row0[e.seq + 1] == q.row0[e.seq]) ++e.seq;
    e.row0 = q.row0[run[i].first];
    e.rows = q.row0[run[i].end] - e.row0;
    e.before = e.len = run[i].positions;
    e.part0 = call->whole_rows;
    call->whole_rows += e.rows;
    const EntryRef at = build.add(e);
    for (int k = run[i].first; k < run[i].end; ++k) {
      common[k] = run[i].positions;
      over[k] = at;
    }
  }
  // behind the shared positions (the longest entries), sequences that write the output, then those of runs
  int order[kMaxSeqs];
  const int n = by_length(q, order);
  for (int pass = 0; pass < 2; ++pass) {
    for (int k = 0; k < n; ++k) {
      const int s = order[k];
      if ((common[s] > 0) != (pass == 1)) continue;
      SpanEntry e = entry_of(q, s);
      if (pass == 0) {
        build.add(e);
        continue;
      }
      e.from = common[s];
      e.part0 = call->whole_rows;
      call->whole_rows += e.rows;
      JoinSeq& j = call->join[call->joins++];
      j.own = build.add(e);
      j.over = over[s];
    }
  }
  if (!build.finish(q)) return false;
  // each unit and KV head of a joined sequence is a block's work of the second kernel
  int64_t jobs = 0;
  for (int k = 0; k < call->joins; ++k) {
    call->join[k].job0 = static_cast<int32_t>(jobs);
    const SpanEntry& e = call->plan[call->join[k].own.kind].e[call->join[k].own.entry];
    jobs += static_cast<int64_t>(e.units) * c.num_kv_heads;
  }
  call->jobs = static_cast<int32_t>(jobs);
  return jobs < (int64_t(1) << 31);
}

}  // namespace mk
