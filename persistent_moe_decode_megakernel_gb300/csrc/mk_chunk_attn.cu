// mk_chunk_attn.cu -- causal attention of a chunk of new tokens over the paged KV cache
// (mk_chunk_attention): which sequences are staged, the launches, the entry points.  The kernels are in
// mk_chunk_attn.cuh.

#include "mk_chunk_attn.cuh"
#include "mk_debug.h"

namespace mk {
namespace {

// Sequences whose cache is staged: from kStageUnits units on decoding once is less work than every unit's block
// doing it (a tile staged costs its bytes, 0.017 us of the card a KV head; a unit's block that decodes
// takes 0.8 us longer a tile, 0.005 us of the card); kStageBytes at most are staged in a call.
constexpr int kStageUnits = 6;
constexpr size_t kStageBytes = size_t(1) << 30;

struct CallPlan {
  AttnPlan direct, staged;           // the two launches' (q8_0 only: staged.items may be 0, as direct.items)
  StageTiles tiles;
  int32_t stage0[kMaxSeqs];
  size_t stage_bytes, floats;        // workspace: staged tiles, then (floats) partials and folds (the launches follow each other)
  size_t direct_folds, staged_folds;
  size_t bytes() const { return stage_bytes + (floats + std::max(direct_folds, staged_folds)) * sizeof(float); }
};

bool plan_call(const mk_cache_shape& c, const ChunkSeqs& q, CallPlan* cp) {
  bool direct[kMaxSeqs], staged[kMaxSeqs];
  cp->stage_bytes = 0;
  cp->tiles.n = 0;
  cp->tiles.first[0] = 0;
  const int UT = 2 * (kTile / (c.num_q_heads / c.num_kv_heads));
  const size_t tile_bytes = static_cast<size_t>(2) * c.num_kv_heads * kTile * c.head_dim * 2;
  for (int s = 0; s < q.n; ++s) {
    const int chunk = q.row0[s + 1] - q.row0[s], tiles = (q.len[s] + kTile - 1) / kTile;
    staged[s] = (c.flags & MK_FLAG_KV_Q8) && (chunk + UT - 1) / UT >= kStageUnits &&
                cp->stage_bytes + tiles * tile_bytes <= kStageBytes;
    direct[s] = !staged[s];
    cp->stage0[s] = 0;
    if (!staged[s]) continue;
    StageTiles& t = cp->tiles;
    cp->stage0[s] = t.first[t.n];
    t.seq[t.n] = s;
    t.first[t.n + 1] = t.first[t.n] + tiles;
    ++t.n;
    cp->stage_bytes += tiles * tile_bytes;
  }
  size_t a = 0, b = 0;
  if (!make_plan(c, q, direct, &cp->direct, &a) || !make_plan(c, q, staged, &cp->staged, &b)) return false;
  cp->floats = std::max(a, b);
  cp->direct_folds = fold_floats(cp->direct, q, c.head_dim);
  cp->staged_folds = fold_floats(cp->staged, q, c.head_dim);
  return true;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_chunk_attention_workspace(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                            const int32_t* seq_lens, size_t* bytes_out) {
  ChunkSeqs seqs;
  const int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (rc) return rc;
  if (!bytes_out) return chunk_fail(MK_ERR_INVALID_ARG, "bytes_out is NULL");
  CallPlan plan;
  if (!plan_call(*shape, seqs, &plan)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  *bytes_out = plan.bytes();
  return MK_OK;
}

extern "C" int mk_chunk_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                  const int32_t* seq_lens, const int32_t* block_tables, const void* q,
                                  int64_t q_stride, const void* kv_layer, void* out, void* workspace,
                                  size_t workspace_bytes, int32_t* status_out, mk_stream_t stream) {
  Params<AttnPlan> p;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &p.seqs);
  if (rc) return rc;
  const mk_cache_shape& c = *shape;
  CallPlan plan;
  if (!plan_call(c, p.seqs, &plan)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  rc = check_attention(c, p.seqs, block_tables, q, q_stride, kv_layer, out, workspace, workspace_bytes, plan.bytes());
  if (rc) return rc;
  const int rows = p.seqs.row0[num_seqs];
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  const bool q8 = (c.flags & MK_FLAG_KV_Q8) != 0;
  fill_params(c, block_tables, q, q_stride, kv_layer, out, status_out, &p);
  p.box = std::min(c.page_size & -c.page_size, kTile);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.stage_bytes);
  std::copy(plan.stage0, plan.stage0 + kMaxSeqs, p.stage0);
  cudaError_t e = cudaSuccess;
  if (plan.direct.items > 0) {
    p.plan = plan.direct;
    p.folds = plan.direct_folds ? p.part + plan.floats : nullptr;
    const bool few = q8 && p.plan.urows <= kFew;
    rc = encode_queries(c, p.plan.G, few ? kFew / p.plan.G : p.plan.TT, q, q_stride, rows, &p.qmap);
    if (rc) return rc;
    if (!q8) {
      rc = encode_pages(c.head_dim, c.num_kv_heads, c.page_size, c.num_pages, true, kv_layer, p.box, &p.map);
      if (rc) return rc;
    }
    e = few                 ? launch_merged<128, kQ8Few>(p, st)
        : q8                ? launch_merged<128, kQ8>(p, st)
        : c.head_dim == 128 ? launch_merged<128, kBf16>(p, st)
                            : launch_merged<64, kBf16>(p, st);
  }
  if (e == cudaSuccess && plan.staged.items > 0) {
    p.plan = plan.staged;
    p.folds = plan.staged_folds ? p.part + plan.floats : nullptr;
    rc = encode_queries(c, p.plan.G, p.plan.TT, q, q_stride, rows, &p.qmap);
    if (!rc) rc = encode_pages(128, c.num_kv_heads, kTile, plan.tiles.first[plan.tiles.n], false, workspace, kTile, &p.map);
    if (rc) return rc;
    stage_kernel<128><<<dim3(plan.tiles.first[plan.tiles.n], 2 * c.num_kv_heads), kStageThreads, 0, st>>>(
        p, static_cast<__half*>(workspace), plan.tiles);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_merged<128, kStaged>(p, st);
  }
  return e == cudaSuccess ? MK_OK : chunk_fail(MK_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
}

extern "C" int mk_plan_chunk_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                       const int32_t* seq_lens, int32_t* segments, int32_t max_segments,
                                       int32_t* n_out) {
  ChunkSeqs seqs;
  const int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (rc) return rc;
  if (!n_out || (max_segments > 0 && !segments)) return chunk_fail(MK_ERR_INVALID_ARG, "NULL output");
  CallPlan plan;
  if (!plan_call(*shape, seqs, &plan)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  int32_t n = 0;
  for (int launch = 0; launch < 2; ++launch) {
    const AttnPlan& pl = launch ? plan.staged : plan.direct;
    for (int b = 0; b < pl.blocks; ++b) {
      SegmentWalk walk(pl, b);
      Segment g;
      while (walk.next(pl, seqs, g)) {
        if (n < max_segments) {
          const int32_t row[9] = {launch, b, g.s, g.unit, g.kvh, g.tile0, g.n, g.tiles, g.slot};
          std::copy(row, row + 9, segments + 9 * static_cast<size_t>(n));
        }
        ++n;
      }
    }
  }
  *n_out = n;
  return MK_OK;
}
