// mk_span_attn.cu -- attention over parts of the paged KV cache: mk_window_attention and mk_prefix_attention.
// The tiles' kernels are those of mk_chunk_attn.cuh over the places of mk_span_plan.h; here are the kernel that joins the
// rows of groups, the launches and the entry points.

#include "mk_chunk_attn.cuh"
#include "mk_debug.h"

namespace mk {
namespace {

// The rows of groups: each has the partials of its own sequence's positions and of the shared ones, in one piece or cut
// over blocks.  A block takes 8 rows of a unit of the sequence's, a thread 4 columns of one; a warp's 8 rows lie side by
// side in a partial.  Sums go over the partials of the sequence, then over those of the group, each in block order.
template <int KINDS>
struct Joins {
  SpanPlan plan[KINDS];
  const float* part[KINDS];
  int32_t n;
  JoinSeq join[kMaxSeqs];
};
struct PartSet {                     // the partials of one row: `first`, then next, next + step, ..
  const float *first, *next;
  size_t step;
  int32_t n, stride, row;
  __device__ __forceinline__ const float* at(int k) const { return k == 0 ? first : next + (k - 1) * step; }
};
template <int D>
__device__ __forceinline__ PartSet parts_of(const Params<SpanPlan>& p, const SpanPlan& pl, const float* part, int entry, int unit,
                                            int kvh, int row) {
  const SpanEntry& e = pl.e[entry];
  const int item = e.item0 + (e.units - 1 - unit) * pl.Hkv + kvh, tok0 = unit * 2 * pl.TT;
  PartSet s;
  s.row = row;
  s.n = 1;
  int b = 0;
  if (pl.ranged) {
    // the first block whose range ends behind the item's beginning, and those whose ranges end inside it
    int lo = 0, hi = pl.blocks - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      const auto end = pl.start[mid + 1];
      if (end.item > item || (end.item == item && end.tile > 0)) hi = mid;
      else lo = mid + 1;
    }
    b = lo;
    while (b + s.n <= pl.blocks && pl.start[b + s.n].item == item) ++s.n;
  }
  if (s.n == 1) {
    s.stride = min(e.rows - tok0, 2 * pl.TT) * pl.G;
    s.first = s.next = p.whole + (static_cast<size_t>(e.part0 + tok0) * p.Hq + static_cast<size_t>(kvh) * s.stride) * (D + 4);
    s.step = 0;
  } else {
    const size_t slot = static_cast<size_t>(pl.urows) * (D + 4);
    s.stride = pl.urows;
    s.first = part + (2 * static_cast<size_t>(b) + 1) * slot;
    s.next = part + 2 * (static_cast<size_t>(b) + 1) * slot;
    s.step = 2 * slot;
  }
  return s;
}

template <int D, int M, int KINDS>
__global__ void __launch_bounds__(2 * D) join_kernel(const __grid_constant__ Params<SpanPlan> p,
                                                     const __grid_constant__ Joins<KINDS> a) {
  constexpr int kRows = 8, kWarps = 2 * D / 32, kMost = 2 * kMaxBlocks;
  __shared__ PartSet sets[kRows][2];
  __shared__ float fac[kRows][kMost], den[kRows];
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.join[mid].job0 <= static_cast<int>(blockIdx.x)) lo = mid;
    else hi = mid;
  }
  const JoinSeq& j = a.join[lo];
  const SpanPlan &own = a.plan[j.own.kind], &over = a.plan[j.over.kind];
  const SpanEntry &e = own.e[j.own.entry], &o = over.e[j.over.entry];
  const int G = own.G, UT = 2 * own.TT, rem = blockIdx.x - j.job0, unit = rem / own.Hkv, kvh = rem - unit * own.Hkv;
  const int rows = min(e.rows - unit * UT, UT) * G, row0 = blockIdx.y * kRows;
  if (row0 >= rows) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < kRows; r += kWarps) {
    const int row = min(row0 + r, rows - 1);
    if (lane < 2) {
      if (lane == 0) {
        sets[r][0] = parts_of<D>(p, own, a.part[j.own.kind], j.own.entry, unit, kvh, row);
      } else {
        const int tok = e.row0 + unit * UT + row / G - o.row0, ou = tok / UT;
        sets[r][1] = parts_of<D>(p, over, a.part[j.over.kind], j.over.entry, ou, kvh, (tok - ou * UT) * G + row % G);
      }
    }
    __syncwarp();
    const int n0 = sets[r][0].n, n = n0 + sets[r][1].n;
    auto ml = [&](int k) {
      const PartSet& s = sets[r][k >= n0];
      return reinterpret_cast<const float2*>(s.at(k >= n0 ? k - n0 : k) + static_cast<size_t>(s.stride) * D)[s.row];
    };
    float top = -INFINITY, L = 0.f;
    for (int k = lane; k < n; k += 32) {
      const float m = ml(k).x;
      fac[r][k] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    for (int k = lane; k < n; k += 32) {
      const float m = fac[r][k], f = m == -INFINITY ? 0.f : ex2(m - top);
      fac[r][k] = f;
      L += f * ml(k).y;
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) L += __shfl_xor_sync(~0u, L, w);
    if (lane == 0) den[r] = L;
  }
  __syncthreads();
  const int lrow = lane & 7, chunk = warp * 4 + (lane >> 3), urow = row0 + lrow;
  const bool live = urow < rows;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  int k0 = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const PartSet s = sets[lrow][i];
    const size_t off = (static_cast<size_t>(chunk) * s.stride + s.row) * 4;
#pragma unroll 8
    for (int k = 0; k < s.n; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(s.at(k) + off);
      const float f = fac[lrow][k0 + k];
      acc.x = fmaf(x.x, f, acc.x);
      acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z);
      acc.w = fmaf(x.w, f, acc.w);
    }
    k0 += s.n;
  }
  const float L = den[lrow], inv = L == 0.f ? 0.f : 1.0f / L;
  const int tok = urow / G, r = e.row0 + unit * UT + tok, h = kvh * G + urow - tok * G;
  acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (live)
    *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(r) * p.Hq + h) * D + chunk * 4) =
        make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
  // (as in merge_kernel)
  const float big = fmaxf(fmaxf(fabsf(acc.x), fabsf(acc.y)), fmaxf(fabsf(acc.z), fabsf(acc.w)));
  const bool odd = live && (L == 0.f || !(big <= 3.3e38f) || acc.x != acc.x || acc.y != acc.y || acc.z != acc.z || acc.w != acc.w);
  __syncthreads();
  uint32_t done = 0;
  for (uint32_t todo = __ballot_sync(~0u, odd); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1;
    const int rr = __shfl_sync(~0u, r, who), hh = __shfl_sync(~0u, h, who), lr = __shfl_sync(~0u, lrow, who);
    if (!((done >> lr) & 1u)) exact_row<D, M>(p, rr, hh, nullptr);
    done |= 1u << lr;
  }
}

template <int D, int M, int KINDS>
cudaError_t join(const SpanCall& call, const Params<SpanPlan>& p, const float* const* part, cudaStream_t st) {
  Joins<KINDS> a;
  int most = 0;
  for (int k = 0; k < KINDS; ++k) {
    a.plan[k] = call.plan[k];
    a.part[k] = part[k];
  }
  a.n = call.joins;
  std::copy(call.join, call.join + call.joins, a.join);
  for (int k = 0; k < call.joins; ++k) {
    const SpanPlan& pl = call.plan[call.join[k].own.kind];
    most = std::max(most, std::min(pl.e[call.join[k].own.entry].rows, 2 * pl.TT) * pl.G);
  }
  join_kernel<D, M, KINDS><<<dim3(call.jobs, (most + 7) / 8), 2 * D, 0, st>>>(p, a);
  return cudaGetLastError();
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
  const bool q8 = (c.flags & MK_FLAG_KV_Q8) != 0;
  fill_params(c, block_tables, q, q_stride, kv_layer, out, status_out, &p);
  p.box = span_box(c);
  float* floats = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + call.stage_bytes);
  p.whole = floats + call.whole0;
  const float* part[kRowKinds];
  cudaError_t e = cudaSuccess;
  for (int k = 0; k < kRowKinds && e == cudaSuccess; ++k) {
    part[k] = floats + call.part0[k];
    if (call.plan[k].items == 0) continue;
    p.plan = call.plan[k];
    p.part = floats + call.part0[k];
    rc = encode_queries(c, p.plan.G, k == kFewRows ? kFew / p.plan.G : p.plan.TT, q, q_stride, rows, &p.qmap);
    if (!rc && k == kStagedRows) rc = encode_pages(128, c.num_kv_heads, kTile, call.stage_tiles, false, workspace, p.box, &p.map);
    if (!rc && !q8) rc = encode_pages(c.head_dim, c.num_kv_heads, c.page_size, c.num_pages, true, kv_layer, p.box, &p.map);
    if (rc) return rc;
    if (k == kStagedRows) {
      StageTiles t;
      t.n = call.staged;
      for (int i = 0; i < t.n; ++i) {
        t.seq[i] = call.tiles_entry[i];
        t.first[i] = p.plan.e[t.seq[i]].stage0;
      }
      t.first[t.n] = call.stage_tiles;
      stage_kernel<128><<<dim3(call.stage_tiles, 2 * c.num_kv_heads), kStageThreads, 0, st>>>(
          p, static_cast<__half*>(workspace), t);
      e = cudaGetLastError();
      if (e == cudaSuccess) e = launch<128, kStaged>(p, st);
    } else {
      e = k == kFewRows       ? launch<128, kQ8Few>(p, st)
          : q8                ? launch<128, kQ8>(p, st)
          : c.head_dim == 128 ? launch<128, kBf16>(p, st)
                              : launch<64, kBf16>(p, st);
    }
  }
  if (e == cudaSuccess && call.joins > 0)
    e = q8                  ? join<128, kQ8, kRowKinds>(call, p, part, st)
        : c.head_dim == 128 ? join<128, kBf16, 1>(call, p, part, st)
                            : join<64, kBf16, 1>(call, p, part, st);
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
