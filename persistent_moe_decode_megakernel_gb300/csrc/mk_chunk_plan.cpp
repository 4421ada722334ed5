// mk_chunk_plan.cpp -- the schedule of mk_chunk_attention (see mk_chunk_plan.h).  Host only.

#include "mk_chunk_plan.h"

#include <algorithm>

#include "mk_schedule.h"

namespace mk {

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
  // visits the items in order: (item, its position tiles, its kind)
  auto each = [&](auto&& visit) {
    int item = 0;
    for (int i = 0; i < pl->n; ++i) {
      const int s = pl->seq[i], chunk = q.row0[s + 1] - q.row0[s], before = q.len[s] - chunk;
      for (int u = pl->units[i] - 1; u >= 0; --u) {
        const int end = std::min(chunk, (u + 1) * UT), t = (before + end - 1) / kTile + 1;
        const int kind = end - u * UT > pl->TT ? kTwoTiles : kOneTile;
        for (int h = 0; h < pl->Hkv; ++h) visit(item++, t, kind);
      }
    }
  };
  schedule(pl, most > pl->TT, c.head_dim, floats, each, [](int) { return true; });
  return true;
}

}  // namespace mk
