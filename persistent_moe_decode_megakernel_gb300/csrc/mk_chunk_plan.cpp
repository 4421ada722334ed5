// mk_chunk_plan.cpp -- the schedule of mk_chunk_attention (see mk_chunk_plan.h).  Host only.

#include "mk_chunk_plan.h"

#include <algorithm>

#include "mk_debug.h"

namespace mk {

namespace {
// Costs in position tiles: what an item adds besides its tiles (query rows in, the pipeline's
// first scores, the epilogue), what a range's partials and the second kernel add, and the fewest
// tiles a block is worth.
constexpr int kItemCost = 2, kMergeCost = 5, kMinRange = 3;
constexpr int kMaxWalk = 16 * kMaxBlocks;   // items beyond which whole ones are even enough
}  // namespace

bool make_plan(const mk_cache_shape& c, const ChunkSeqs& q, AttnPlan* pl, size_t* floats) {
  pl->Hkv = c.num_kv_heads;
  pl->G = c.num_q_heads / c.num_kv_heads;
  pl->TT = kTile / pl->G;
  pl->by_G = 65536 / pl->G + 1;   // exact below 2^9 rows
  pl->n = pl->items = pl->blocks = pl->ranged = 0;
  *floats = 0;
  const int UT = 2 * pl->TT;
  int most = 0;
  for (int s = 0; s < q.n; ++s) {
    const int chunk = q.row0[s + 1] - q.row0[s];
    if (chunk == 0) continue;
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

  // the slowest block of whole items, and the work altogether
  int64_t load[kMaxBlocks] = {}, tiles = 0;
  Segment g;
  for (int i = 0; i < pl->items; ++i) {
    item_of(*pl, q, i, g);
    tiles += g.tiles;
    const int round = i / pl->blocks, at = i % pl->blocks;
    load[round & 1 ? pl->blocks - 1 - at : at] += g.tiles + kItemCost;
  }
  const int64_t whole = *std::max_element(load, load + pl->blocks);
  const int nb = static_cast<int>(std::min<int64_t>(kMaxBlocks, (tiles + kMinRange - 1) / kMinRange));
  const int64_t cost = tiles + items * kItemCost;
  if (whole <= (cost + nb - 1) / nb + kMergeCost) return true;

  // cut the line of items (each kItemCost, then its tiles) at equal cost
  pl->ranged = 1;
  pl->blocks = nb;
  int b = 1;
  int64_t at = 0;   // cost before item i
  pl->start[0] = {0, 0};
  for (int i = 0; i < pl->items; ++i) {
    item_of(*pl, q, i, g);
    const int64_t end = at + kItemCost + g.tiles;
    for (; b < nb; ++b) {
      const int64_t x = cost * b / nb;
      if (x >= end) break;
      const int64_t t = x - at - kItemCost;
      if (t < 1) pl->start[b] = {i, 0};
      else pl->start[b] = {i, static_cast<int32_t>(t)};   // 1 <= t < tiles
    }
    at = end;
  }
  for (; b <= nb; ++b) pl->start[b] = {pl->items, 0};
  *floats = static_cast<size_t>(2) * nb * pl->urows * (c.head_dim + 4);
  return true;
}

}  // namespace mk

using namespace mk;

extern "C" int mk_plan_chunk_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                       const int32_t* seq_lens, int32_t* segments, int32_t max_segments,
                                       int32_t* n_out) {
  ChunkSeqs seqs;
  const int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (rc) return rc;
  if (!n_out || (max_segments > 0 && !segments)) return chunk_fail(MK_ERR_INVALID_ARG, "NULL output");
  AttnPlan plan;
  size_t floats = 0;
  if (!make_plan(*shape, seqs, &plan, &floats)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  int32_t n = 0;
  for (int b = 0; b < plan.blocks; ++b) {
    SegmentWalk walk(plan, b);
    Segment g;
    while (walk.next(plan, seqs, g)) {
      if (n < max_segments) {
        const int32_t row[8] = {b, g.s, g.unit, g.kvh, g.tile0, g.n, g.tiles, g.slot};
        std::copy(row, row + 8, segments + 8 * static_cast<size_t>(n));
      }
      ++n;
    }
  }
  *n_out = n;
  return MK_OK;
}
