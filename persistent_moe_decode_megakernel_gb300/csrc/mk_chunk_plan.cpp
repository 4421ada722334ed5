// mk_chunk_plan.cpp -- the schedule of mk_chunk_attention (see mk_chunk_plan.h).  Host only.

#include "mk_chunk_plan.h"

#include <algorithm>

namespace mk {

namespace {
// Costs in tenths of a microsecond, as measured: a position tile and what an item adds to its tiles
// (query rows, the pipeline's filling and emptying, the epilogue), for items of two tiles of rows and
// of one; what the ranges' partials and the second kernel add (more where units of two tiles are cut:
// an 8192-token prompt, even to 1 % as whole items, took 383 us so and 393 us in ranges).  (152 blocks streaming from HBM.)
constexpr int kTileCost[2] = {14, 17}, kItemCost[2] = {40, 60}, kMergeCost[2] = {80, 250};
constexpr int kMinRange = 3;                // position tiles a block is worth
constexpr int kMaxWalk = 1 << 17;            // items beyond which whole ones are even enough (and the walk long)
}  // namespace

bool make_plan(const mk_cache_shape& c, const ChunkSeqs& q, const bool* use, AttnPlan* pl, size_t* floats) {
  pl->Hkv = c.num_kv_heads;
  pl->G = c.num_q_heads / c.num_kv_heads;
  pl->TT = kTile / pl->G;
  pl->by_G = 65536 / pl->G + 1;   // exact below 2^9 rows
  pl->n = pl->items = pl->blocks = pl->ranged = pl->cuts = 0;
  *floats = 0;
  const int UT = 2 * pl->TT;
  int most = 0;
  for (int s = 0; s < q.n; ++s) {
    const int chunk = q.row0[s + 1] - q.row0[s];
    if (chunk == 0 || !use[s]) continue;
    pl->seq[pl->n++] = s;
    most = std::max(most, std::min(chunk, UT));
  }
  pl->urows = most * pl->G;
  std::sort(pl->seq, pl->seq + pl->n,
            [&](int a, int b) { return q.len[a] != q.len[b] ? q.len[a] > q.len[b] : a < b; });
  int64_t items = 0;
  for (int i = 0; i < pl->n; ++i) {
    const int s = pl->seq[i], chunk = q.row0[s + 1] - q.row0[s];
    pl->item0[i] = static_cast<int32_t>(items);
    pl->units[i] = (chunk + UT - 1) / UT;
    items += static_cast<int64_t>(pl->units[i]) * pl->Hkv;
    if (items >= (int64_t(1) << 31)) return false;
  }
  pl->item0[pl->n] = static_cast<int32_t>(items);
  pl->items = static_cast<int32_t>(items);
  pl->blocks = static_cast<int32_t>(std::min<int64_t>(items, kMaxBlocks));
  if (items == 0 || items > kMaxWalk) return true;

  // visits the items in order: (item, its position tiles, whether it has two tiles of rows)
  auto each = [&](auto&& visit) {
    int item = 0;
    for (int i = 0; i < pl->n; ++i) {
      const int s = pl->seq[i], chunk = q.row0[s + 1] - q.row0[s], before = q.len[s] - chunk;
      for (int u = pl->units[i] - 1; u >= 0; --u) {
        const int end = std::min(chunk, (u + 1) * UT), t = (before + end - 1) / kTile + 1;
        const bool two = end - u * UT > pl->TT;
        for (int h = 0; h < pl->Hkv; ++h) visit(item++, t, two);
      }
    }
  };
  // the slowest block of whole items, and the work altogether
  int64_t load[kMaxBlocks] = {}, tiles = 0, cost = 0;
  int at_block = 0, step = 1;
  each([&](int, int t, bool two) {
    const int64_t x = t * kTileCost[two] + kItemCost[two];
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
  if (whole <= (cost + nb - 1) / nb + kMergeCost[most > pl->TT]) return true;

  // cut the line of items (each its own cost, then its tiles') at equal cost
  pl->ranged = 1;
  pl->blocks = nb;
  int b = 1;
  int64_t at = 0;   // cost before item i
  pl->start[0] = {0, 0};
  each([&](int item, int t, bool two) {
    const int64_t end = at + kItemCost[two] + t * kTileCost[two];
    for (; b < nb; ++b) {
      const int64_t x = cost * b / nb;
      if (x >= end) break;
      // (x within the item's own cost: the cut is before it; else after 0 <= . < t of its tiles)
      const int64_t cut = x < at + kItemCost[two] ? 0 : (x - at - kItemCost[two]) / kTileCost[two];
      pl->start[b] = {item, static_cast<int32_t>(cut)};
    }
    at = end;
  });
  for (; b <= nb; ++b) pl->start[b] = {pl->items, 0};
  for (b = 0; b < nb; ++b) {
    const int item = pl->start[b + 1].item;
    if (pl->start[b + 1].tile == 0 || (pl->start[b].item == item && pl->start[b].tile > 0)) continue;
    int n = 2;
    while (b + n <= nb && pl->start[b + n].item == item) ++n;
    pl->cut_block[pl->cuts] = static_cast<uint8_t>(b);
    pl->cut_parts[pl->cuts++] = static_cast<uint8_t>(n);
  }
  *floats = static_cast<size_t>(2) * nb * pl->urows * (c.head_dim + 4);
  return true;
}

}  // namespace mk
