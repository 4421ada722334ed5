// mk_schedule.h -- how the items of an attention launch are dealt out over the blocks (host only): whole items in
// alternating order, or one range of position tiles a block (see mk_chunk_plan.h).
#ifndef MK_SCHEDULE_H
#define MK_SCHEDULE_H

#include <algorithm>

#include "mk_chunk_plan.h"

namespace mk {

// Costs in tenths of a microsecond, as measured: a position tile and what an item adds to its tiles
// (query rows, the pipeline's filling and emptying, the epilogue), for items of one tile of rows and, second, of
// two; what the ranges' partials and the second kernel add (more where units of two tiles are cut:
// an 8192-token prompt, even to 1 % as whole items, took 383 us so and 393 us in ranges).  (152 blocks streaming from HBM.)
// Third, items of two KV heads: both heads' tiles.
enum { kOneTile, kTwoTiles, kTwoHeads };
constexpr int kTileCost[3] = {14, 17, 28}, kItemCost[3] = {40, 60, 40}, kMergeCost[2] = {80, 250};
constexpr int kMinRange = 3;                // position tiles a block is worth
constexpr int kMaxWalk = 1 << 17;            // items beyond which whole ones are even enough (and the walk long)

// `each` visits the plan's items in order: (item, its position tiles, which of the three kinds it is).  Fills
// ranged, blocks, start and the cut items of which `joined` (item) is true; *floats is the size of their partials.
template <class Plan, class Each, class Joined>
void schedule(Plan* pl, bool any_two, int head_dim, size_t* floats, Each&& each, Joined&& joined) {
  pl->blocks = std::min<int32_t>(pl->items, kMaxBlocks);
  if (pl->items == 0 || pl->items > kMaxWalk) return;
  // the slowest block of whole items, and the work altogether
  int64_t load[kMaxBlocks] = {}, tiles = 0, cost = 0;
  int at_block = 0, step = 1;
  each([&](int, int t, int kind) {
    const int64_t x = t * kTileCost[kind] + kItemCost[kind];
    tiles += t;
    cost += x;
    load[at_block] += x;
    at_block += step;                       // 0..B-1, then B-1..0
    if (at_block == pl->blocks || at_block < 0) {
      step = -step;
      at_block += step;
    }
  });
  const int64_t whole = *std::max_element(load, load + pl->blocks);
  const int nb = static_cast<int>(std::min<int64_t>(kMaxBlocks, (tiles + kMinRange - 1) / kMinRange));
  if (whole <= (cost + nb - 1) / nb + kMergeCost[any_two]) return;

  // cut the line of items (each its own cost, then its tiles') at equal cost
  pl->ranged = 1;
  pl->blocks = nb;
  int b = 1;
  int64_t at = 0;   // cost before item i
  pl->start[0] = {0, 0};
  each([&](int item, int t, int kind) {
    const int64_t end = at + kItemCost[kind] + t * kTileCost[kind];
    for (; b < nb; ++b) {
      const int64_t x = cost * b / nb;
      if (x >= end) break;
      // (x within the item's own cost: the cut is before it; else after 0 <= . < t of its tiles)
      const int64_t cut = x < at + kItemCost[kind] ? 0 : (x - at - kItemCost[kind]) / kTileCost[kind];
      pl->start[b] = {item, static_cast<int32_t>(cut)};
    }
    at = end;
  });
  for (; b <= nb; ++b) pl->start[b] = {pl->items, 0};
  for (b = 0; b < nb; ++b) {
    const int item = pl->start[b + 1].item;
    if (pl->start[b + 1].tile == 0 || (pl->start[b].item == item && pl->start[b].tile > 0)) continue;
    if (!joined(item)) continue;
    int n = 2;
    while (b + n <= nb && pl->start[b + n].item == item) ++n;
    pl->cut_block[pl->cuts] = static_cast<uint8_t>(b);
    pl->cut_parts[pl->cuts++] = static_cast<uint8_t>(n);
  }
  *floats = static_cast<size_t>(2) * nb * pl->urows * (head_dim + 4);
}

}  // namespace mk

#endif
