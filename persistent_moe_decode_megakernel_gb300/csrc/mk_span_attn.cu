// mk_span_attn.cu -- attention over parts of the paged KV cache: mk_window_attention and mk_prefix_attention.

#include "mk_chunk_attn.cuh"
#include "mk_debug.h"

namespace mk {
namespace {

// Every row and query head by a warp (exact_row): right for every call, and the measure of the rest.
template <int D, int M>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ Params<SpanPlan> p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (i >= static_cast<int64_t>(p.seqs.row0[p.seqs.n]) * p.Hq) return;
  const int r = static_cast<int>(i / p.Hq), s = seq_of_row(p.seqs, r), n = p.seqs.len[s] - p.seqs.row0[s + 1] + r + 1;
  exact_row<D, M>(p, r, static_cast<int>(i % p.Hq), nullptr);
  const int lo = max(n - p.plan.window, 0);
  for (int t = threadIdx.x & 31; t < n; t += 32) {
    if (t < lo && t >= p.plan.sinks) continue;
    const int page = __ldg(p.bt + static_cast<size_t>(s) * p.maxpg + t / p.ps);
    if ((page < 0 || page >= p.P) && p.status) *p.status = MK_ERR_DEVICE_BOUNDS;
  }
}

int attend(const mk_cache_shape& c, const SpanCall& call, Params<SpanPlan>& p, const int32_t* block_tables, const void* q,
           int64_t q_stride, const void* kv_layer, void* out, void* workspace, size_t workspace_bytes, int32_t* status_out,
           mk_stream_t stream) {
  int rc = check_attention(c, p.seqs, block_tables, q, q_stride, kv_layer, out, workspace, workspace_bytes, call.bytes());
  if (rc) return rc;
  const int rows = p.seqs.row0[p.seqs.n];
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  fill_params(c, block_tables, q, q_stride, kv_layer, out, status_out, &p);
  p.plan = call.plan[0];
  const int64_t blocks = (static_cast<int64_t>(rows) * c.num_q_heads + 7) / 8;
  if (c.flags & MK_FLAG_KV_Q8) rows_kernel<128, kQ8><<<static_cast<unsigned>(blocks), 256, 0, st>>>(p);
  else if (c.head_dim == 128) rows_kernel<128, kBf16><<<static_cast<unsigned>(blocks), 256, 0, st>>>(p);
  else rows_kernel<64, kBf16><<<static_cast<unsigned>(blocks), 256, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MK_OK : chunk_fail(MK_ERR_CUDA, "attention over parts of the cache: %s", cudaGetErrorString(e));
}

int check_window(int32_t window, int32_t sinks) {
  if (window < 1) return chunk_fail(MK_ERR_INVALID_ARG, "window must be > 0 (got %d)", window);
  if (sinks < 0) return chunk_fail(MK_ERR_INVALID_ARG, "sinks must be >= 0 (got %d)", sinks);
  return MK_OK;
}

int check_groups(const ChunkSeqs& q, int32_t num_groups, const int32_t* group_seqs, const int32_t* prefix_lens) {
  if (num_groups < 1 || num_groups > q.n) return chunk_fail(MK_ERR_INVALID_ARG, "num_groups outside 1..num_seqs");
  if (!group_seqs || !prefix_lens) return chunk_fail(MK_ERR_INVALID_ARG, "group_seqs or prefix_lens is NULL");
  int s = 0;
  for (int i = 0; i < num_groups; ++i) {
    if (group_seqs[i] < 1 || group_seqs[i] > q.n - s)
      return chunk_fail(MK_ERR_INVALID_ARG, "group %d: the groups' sequences do not add up to num_seqs", i);
    if (prefix_lens[i] < 0) return chunk_fail(MK_ERR_INVALID_ARG, "group %d: prefix_len must be >= 0", i);
    for (int k = 0; k < group_seqs[i]; ++k, ++s)
      if (prefix_lens[i] > q.len[s] - (q.row0[s + 1] - q.row0[s]))
        return chunk_fail(MK_ERR_INVALID_ARG, "group %d: prefix_len (%d) reaches into the new tokens of sequence %d", i,
                          prefix_lens[i], s);
  }
  if (s != q.n) return chunk_fail(MK_ERR_INVALID_ARG, "the groups' sequences do not add up to num_seqs");
  return MK_OK;
}

int too_many() { return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call"); }

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_window_attention_workspace(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                             const int32_t* seq_lens, int32_t window, int32_t sinks, size_t* bytes_out) {
  ChunkSeqs seqs;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (!rc) rc = check_window(window, sinks);
  if (rc) return rc;
  if (!bytes_out) return chunk_fail(MK_ERR_INVALID_ARG, "bytes_out is NULL");
  SpanCall call;
  if (!plan_window(*shape, seqs, window, sinks, &call)) return too_many();
  *bytes_out = call.bytes();
  return MK_OK;
}

extern "C" int mk_window_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                   const int32_t* seq_lens, int32_t window, int32_t sinks, const int32_t* block_tables,
                                   const void* q, int64_t q_stride, const void* kv_layer, void* out, void* workspace,
                                   size_t workspace_bytes, int32_t* status_out, mk_stream_t stream) {
  Params<SpanPlan> p;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &p.seqs);
  if (!rc) rc = check_window(window, sinks);
  if (rc) return rc;
  SpanCall call;
  if (!plan_window(*shape, p.seqs, window, sinks, &call)) return too_many();
  return attend(*shape, call, p, block_tables, q, q_stride, kv_layer, out, workspace, workspace_bytes, status_out, stream);
}

extern "C" int mk_prefix_attention_workspace(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                             const int32_t* seq_lens, int32_t num_groups, const int32_t* group_seqs,
                                             const int32_t* prefix_lens, size_t* bytes_out) {
  ChunkSeqs seqs;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (!rc) rc = check_groups(seqs, num_groups, group_seqs, prefix_lens);
  if (rc) return rc;
  if (!bytes_out) return chunk_fail(MK_ERR_INVALID_ARG, "bytes_out is NULL");
  SpanCall call;
  if (!plan_prefix(*shape, seqs, num_groups, group_seqs, prefix_lens, &call)) return too_many();
  *bytes_out = call.bytes();
  return MK_OK;
}

extern "C" int mk_prefix_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                   const int32_t* seq_lens, int32_t num_groups, const int32_t* group_seqs,
                                   const int32_t* prefix_lens, const int32_t* block_tables, const void* q, int64_t q_stride,
                                   const void* kv_layer, void* out, void* workspace, size_t workspace_bytes,
                                   int32_t* status_out, mk_stream_t stream) {
  Params<SpanPlan> p;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &p.seqs);
  if (!rc) rc = check_groups(p.seqs, num_groups, group_seqs, prefix_lens);
  if (rc) return rc;
  SpanCall call;
  if (!plan_prefix(*shape, p.seqs, num_groups, group_seqs, prefix_lens, &call)) return too_many();
  return attend(*shape, call, p, block_tables, q, q_stride, kv_layer, out, workspace, workspace_bytes, status_out, stream);
}

extern "C" int mk_plan_span_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                      const int32_t* seq_lens, int32_t window, int32_t sinks, int32_t num_groups,
                                      const int32_t* group_seqs, const int32_t* prefix_lens, int32_t* segments,
                                      int32_t max_segments, int32_t* n_out) {
  ChunkSeqs seqs;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (!rc) rc = num_groups > 0 ? check_groups(seqs, num_groups, group_seqs, prefix_lens) : check_window(window, sinks);
  if (rc) return rc;
  if (!n_out || (max_segments > 0 && !segments)) return chunk_fail(MK_ERR_INVALID_ARG, "NULL output");
  SpanCall call;
  if (!(num_groups > 0 ? plan_prefix(*shape, seqs, num_groups, group_seqs, prefix_lens, &call)
                       : plan_window(*shape, seqs, window, sinks, &call)))
    return too_many();
  int32_t n = 0;
  for (int k = 0; k < kRowKinds; ++k) {
    const SpanPlan& pl = call.plan[k];
    for (int b = 0; b < pl.blocks; ++b) {
      SegmentWalk walk(pl, b);
      Segment g;
      while (walk.next(pl, seqs, g)) {
        if (n < max_segments) {
          const SpanEntry& e = pl.e[g.entry];
          const int32_t row[18] = {k,     b,       g.entry, g.s,  g.row0,  g.ntok, g.kvh,    g.head,         g.gap,
                                   g.pos0, g.len,  g.tile0, g.n,  g.tiles, g.slot, e.stage0, e.stage_tile0, e.stage_head};
          std::copy(row, row + 18, segments + 18 * static_cast<size_t>(n));
        }
        ++n;
      }
    }
  }
  *n_out = n;
  return MK_OK;
}
