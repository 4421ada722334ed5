// mk_span_attn.cu -- attention over parts of the paged KV cache: mk_window_attention and mk_prefix_attention.
// The tiles' kernels are those of mk_chunk_attn.cuh over the places of mk_span_plan.h; here are the kernel that joins the
// rows of groups, the launches and the entry points.

#include "mk_chunk_attn.cuh"
#include "mk_debug.h"
#include "mk_span_call.h"

namespace mk {
namespace {

// Joins partials: of a cut item's rows (in block order), and of the rows of groups, which have those of their own
// sequence's positions and then those of the shared ones, each in one piece or cut.
//
// 8 rows lie side by side in a partial, so 8 lanes read 128 bytes of one; the warp's other lanes take other columns.
// What it takes is latency.  Few rows: a block's 8 warps take every eighth partial each of 16 columns (kSplit).  More: a warp
// has 16 columns and all partials, 12 of them on their way before it waits for the first, two blocks an SM (kDeep).  Many
// rows: more and lighter blocks, each over several groups of 8 rows (kMany).
//
// The launch brings just what is looked up, and a block copies it into shared memory at once, before it waits for the
// kernel that writes the partials (walked where it lies, in the constant bank, each step of a search was a miss of its
// own).
struct Sight {
  static constexpr bool kSpans = true;
  int32_t G, Hkv, window, sinks;
};
struct JoinParams : CallParams {     // what the rows that are worked out again need
  Sight plan;
};
enum { kSplit, kDeep, kMany };
struct JoinEntry {
  int32_t row0, rows, units, item0, part0;
  int8_t kind, pair;
  int16_t pad;
};
template <int KINDS>
struct alignas(16) Joins {
  // of each launch: where its blocks' ranges begin, item * 2 + whether inside the item (whole items: no block)
  int32_t start[KINDS][kMaxBlocks + 1], blocks[KINDS], urows[KINDS];
  const float* part[KINDS];
  const float* whole;
  int32_t cuts, n, Hkv, G, UT, pad;
  struct { JoinEntry own, over; int32_t job0, pad; } join[kMaxSeqs];   // sequences of groups
  struct { int32_t row0; int16_t rows, kvh; uint8_t kind, pair, block, parts; } cut[KINDS * kMaxBlocks];   // cut items
};
struct PartSet {                     // the partials of one row: `first`, then next, next + step, ..
  const float *first, *next;
  size_t step;
  int32_t n, stride, row;
  __device__ __forceinline__ const float* at(int k) const { return k == 0 ? first : next + (k - 1) * step; }
  template <int D>
  __device__ __forceinline__ float2 ml(int k) const {
    return reinterpret_cast<const float2*>(at(k) + static_cast<size_t>(stride) * D)[row];
  }
  __device__ __forceinline__ const float4* address(int k, int chunk) const {
    return reinterpret_cast<const float4*>(at(k)) + static_cast<size_t>(chunk) * stride + row;
  }
  __device__ __forceinline__ float4 columns(int k, int chunk) const { return *address(k, chunk); }
};
// of a cut item that block b begins
template <int D, int KINDS>
__device__ __forceinline__ PartSet cut_parts(const Joins<KINDS>& a, int kind, int b, int n, int row) {
  const size_t slot = static_cast<size_t>(a.urows[kind]) * (D + 4);
  PartSet s;
  s.n = n;
  s.row = row;
  s.stride = a.urows[kind];
  s.first = a.part[kind] + (2 * static_cast<size_t>(b) + 1) * slot;
  s.next = a.part[kind] + 2 * (static_cast<size_t>(b) + 1) * slot;
  s.step = 2 * slot;
  return s;
}
template <int D, int KINDS>
__device__ __forceinline__ PartSet parts_of(const Joins<KINDS>& a, const JoinEntry& e, int unit, int kvh, int row) {
  const int item = e.item0 + (e.units - 1 - unit) * (a.Hkv >> e.pair) + (kvh >> e.pair), tok0 = unit * a.UT;
  const int blocks = a.blocks[e.kind], rows = min(e.rows - tok0, a.UT) * a.G;
  const int32_t* start = a.start[e.kind];
  int n = 1, b = 0;
  if (blocks > 0) {
    // the first block whose range ends behind the item's beginning, and those whose ranges end inside it
    int hi = blocks - 1;
    while (b < hi) {
      const int mid = (b + hi) >> 1;
      if (start[mid + 1] > 2 * item) hi = mid;
      else b = mid + 1;
    }
    while (b + n <= blocks && start[b + n] == 2 * item + 1) ++n;
  }
  if (n > 1) return cut_parts<D>(a, e.kind, b, n, row + (kvh & e.pair) * rows);
  PartSet s;
  s.n = 1;
  s.row = row;
  s.stride = rows;
  s.first = s.next = a.whole + (static_cast<size_t>(e.part0 + tok0) * a.G * a.Hkv + static_cast<size_t>(kvh) * rows) * (D + 4);
  s.step = 0;
  return s;
}

template <int D, int M, int KINDS, int kMode>
__global__ void __launch_bounds__(kMode == kSplit ? 256 : 2 * D, kMode == kSplit ? 3 : kMode == kDeep ? 256 / D : 512 / D)
    join_kernel(const __grid_constant__ JoinParams p, const __grid_constant__ Joins<KINDS> given) {
  constexpr int kThreads = kMode == kSplit ? 256 : 2 * D, kAhead = kMode == kSplit ? 5 : kMode == kDeep ? 12 : 3;
  constexpr int kEvery = kMode == kSplit ? 8 : 1;
  __shared__ Joins<KINDS> a;
  __shared__ PartSet sets[2][8][2];
  // (by their generic address: constant reads would go one lane at a time; and all at once)
  constexpr int kWords = sizeof a / 16, kReads = (kWords + kThreads - 1) / kThreads;
  uint4 w[kReads];
#pragma unroll
  for (int i = 0; i < kReads; ++i) {
    const int at = min(static_cast<int>(threadIdx.x) + i * kThreads, kWords - 1);
    asm volatile("ld.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                 : "l"(reinterpret_cast<const uint4*>(&given) + at));
  }
#pragma unroll
  for (int i = 0; i < kReads; ++i)
    reinterpret_cast<uint4*>(&a)[min(static_cast<int>(threadIdx.x) + i * kThreads, kWords - 1)] = w[i];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.G, UT = a.UT;
  const int chunk = (kMode == kSplit ? static_cast<int>(blockIdx.z) : warp) * 4 + (lane >> 3), mine = kMode == kSplit ? warp : 0;
  const bool cut = static_cast<int>(blockIdx.x) < a.cuts;
  int lo = 0, unit = 0, kvh, hrows, rows, r0;
  if (cut) {
    const auto& c = a.cut[blockIdx.x];
    kvh = c.kvh;
    hrows = c.rows * G;
    rows = hrows << c.pair;
    r0 = c.row0;
  } else {
    const int job = blockIdx.x - a.cuts;
    int hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.join[mid].job0 <= job) lo = mid;
      else hi = mid;
    }
    const JoinEntry& e = a.join[lo].own;
    const int rem = job - a.join[lo].job0;
    unit = rem / a.Hkv;
    kvh = rem - unit * a.Hkv;
    hrows = rows = min(e.rows - unit * UT, UT) * G;
    r0 = e.row0 + unit * UT;
  }
  // where a group of 8 rows finds its partials: 16 lanes of one warp look it up, a group ahead
  auto find = [&](int row0, int into) {
    if (warp != 0 || lane >= 16) return;
    const int row = min(row0 + (lane & 7), rows - 1), over = lane >> 3;
    if (cut) {
      const auto& c = a.cut[blockIdx.x];
      sets[into][lane & 7][over] = cut_parts<D>(a, c.kind, c.block, c.parts, row);
      if (over) sets[into][lane & 7][over].n = 0;
    } else {
      const JoinEntry& o = a.join[lo].over;
      const int tok = row / G, ot = r0 + tok - o.row0, ou = ot / UT;
      sets[into][lane & 7][over] = over ? parts_of<D>(a, o, ou, kvh, (ot - ou * UT) * G + row - tok * G)
                                        : parts_of<D>(a, a.join[lo].own, unit, kvh, row);
    }
  };
  int row0 = blockIdx.y * 8, turn = 0;
  if (row0 >= rows) return;
  find(row0, 0);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (; row0 < rows; row0 += gridDim.y * 8, turn ^= 1) {
    const bool live = row0 + (lane & 7) < rows;
    const int row = min(row0 + (lane & 7), rows - 1), second = row >= hrows ? 1 : 0, hrow = row - second * hrows;
    const int tok = hrow / G, r = r0 + tok, h = (kvh + second) * G + hrow - tok * G;
    const PartSet &own = sets[turn][lane & 7][0], &over = sets[turn][lane & 7][1];
    const int n = own.n + over.n;    // partials, the own ones first
    auto ml = [&](int k) { return k < own.n ? own.template ml<D>(k) : over.template ml<D>(k - own.n); };
    auto columns = [&](int k) { return k < own.n ? own.columns(k, chunk) : over.columns(k - own.n, chunk); };
    float4 held[kAhead];
    float2 held_ml[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = mine + i * kEvery;
      held_ml[i] = k < n ? ml(k) : make_float2(-INFINITY, 0.f);
      held[i] = k < n ? columns(k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if constexpr (kMode == kDeep)
      for (int k = kAhead; k < n; ++k)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(k < own.n ? own.address(k, chunk) : over.address(k - own.n, chunk)));
    find(row0 + gridDim.y * 8, turn ^ 1);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) top = fmaxf(top, held_ml[i].x);
#pragma unroll 8
    for (int k = mine + kAhead * kEvery; k < n; k += kEvery) top = fmaxf(top, ml(k).x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    auto add = [&](const float4 x, const float2 ml) {
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      L = fmaf(ml.y, f, L);
      acc.x = fmaf(x.x, f, acc.x);
      acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z);
      acc.w = fmaf(x.w, f, acc.w);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) add(held[i], held_ml[i]);
#pragma unroll 8
    for (int k = mine + kAhead * kEvery; k < n; k += kEvery) add(columns(k), ml(k));
    if constexpr (kMode == kSplit) {
      // the warps' sums, each relative to its own maximum, in the warps' order
      __shared__ float4 sums[8][32];
      __shared__ float2 scale[8][32];
      sums[warp][lane] = acc;
      scale[warp][lane] = make_float2(top, L);
      __syncthreads();
      top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 8; ++w) top = fmaxf(top, scale[w][lane].x);
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      L = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) add(sums[w][lane], scale[w][lane]);
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (live && mine == 0)
      *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(r) * p.Hq + h) * D + chunk * 4) =
          make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
    // (as in merge_kernel; a row's columns are several warps')
    const float big = fmaxf(fmaxf(fabsf(acc.x), fabsf(acc.y)), fmaxf(fabsf(acc.z), fabsf(acc.w)));
    const bool odd = live && mine == 0 && (L == 0.f || !(big <= 3.3e38f) || acc.x != acc.x || acc.y != acc.y || acc.z != acc.z || acc.w != acc.w);
    if (__syncthreads_or(odd)) {
      uint32_t done = 0;
      for (uint32_t todo = __ballot_sync(~0u, odd); todo; todo &= todo - 1) {
        const int who = __ffs(todo) - 1, lr = who & 7;
        const int rr = __shfl_sync(~0u, r, who), hh = __shfl_sync(~0u, h, who);
        // (a split row's columns are several blocks': each writes its own, so that no two results of a value meet)
        if (!((done >> lr) & 1u)) exact_row<D, M, kMode == kSplit ? 16 : D>(p, rr, hh, nullptr, kMode == kSplit ? blockIdx.z * 16 : 0);
        done |= 1u << lr;
      }
    }
  }
}
template <int D, int M, int KINDS>
cudaError_t join(const SpanCall& call, const Params<SpanPlan>& given, const float* const* part, cudaStream_t st) {
  int cuts = 0;
  for (int k = 0; k < KINDS; ++k) cuts += call.plan[k].items > 0 ? call.plan[k].cuts : 0;
  if (cuts + call.jobs == 0) return cudaSuccess;
  Joins<KINDS> a;
  static_assert(sizeof a % 16 == 0, "");
  const int UT = 2 * call.plan[0].TT, G = call.plan[0].G;
  JoinParams p;                         // what the rows that are worked out again need
  static_cast<CallParams&>(p) = given;
  p.plan.G = G;
  p.plan.Hkv = call.plan[0].Hkv;
  p.plan.window = call.plan[0].window;
  p.plan.sinks = call.plan[0].sinks;
  int most = 0, parts = 0;           // rows of a job, partials of a row
  int64_t groups = 0;                // of 8 rows
  a.cuts = 0;
  for (int k = 0; k < KINDS; ++k) {
    const SpanPlan& pl = call.plan[k];
    a.blocks[k] = pl.items > 0 && pl.ranged ? pl.blocks : 0;
    for (int b = 0; b <= kMaxBlocks; ++b)
      a.start[k][b] = b <= a.blocks[k] && a.blocks[k] ? 2 * pl.start[b].item + (pl.start[b].tile > 0) : 0;
    a.urows[k] = pl.urows;
    a.part[k] = part[k];
    for (int i = 0; i < (pl.items > 0 ? pl.cuts : 0); ++i) {
      Segment g;
      const int item = pl.start[pl.cut_block[i] + 1].item;
      item_of_entry(pl, entry_of_item(pl, item), item, g);
      auto& x = a.cut[a.cuts++];
      x.row0 = g.row0;
      x.rows = static_cast<int16_t>(g.ntok);
      x.kvh = static_cast<int16_t>(g.kvh);
      x.kind = static_cast<uint8_t>(k);
      x.pair = g.pair;
      x.block = pl.cut_block[i];
      x.parts = pl.cut_parts[i];
      const int rows = g.ntok * G << x.pair;
      most = std::max(most, rows);
      groups += (rows + 7) / 8;
      parts = std::max<int>(parts, x.parts);
    }
  }
  a.whole = given.whole;
  a.n = call.joins;
  a.Hkv = call.plan[0].Hkv;
  a.G = G;
  a.UT = UT;
  auto entry = [&](const EntryRef& r) {
    const SpanEntry& e = call.plan[r.kind].e[r.entry];
    return JoinEntry{e.row0, e.rows, e.units, e.item0, e.part0, r.kind, static_cast<int8_t>(e.pair), 0};
  };
  for (int k = 0; k < call.joins; ++k) {
    a.join[k] = {entry(call.join[k].own), entry(call.join[k].over), call.join[k].job0, 0};
    const int rows = std::min(a.join[k].own.rows, UT) * G;
    most = std::max(most, rows);
    groups += static_cast<int64_t>(a.join[k].own.units) * a.Hkv * ((rows + 7) / 8);
    // (the blocks that begin among the group's items, over these)
    const JoinEntry& o = a.join[k].over;
    if (k > 0 && o.row0 == a.join[k - 1].over.row0) continue;
    const int64_t items = static_cast<int64_t>(o.units) * (a.Hkv >> o.pair);
    int64_t in = 0;
    for (int b = 0; b < a.blocks[o.kind]; ++b) in += a.start[o.kind][b] / 2 >= o.item0 && a.start[o.kind][b] / 2 < o.item0 + items;
    parts = std::max<int>(parts, static_cast<int>(2 + in / items));
  }
  const int jobs = a.cuts + call.jobs;
  const dim3 all(jobs, (most + 7) / 8);
  // Calls of 32 / 4 heads of 128, as in mk_span_plan.cpp.  Split and deep: one token through 32768 26 us and 55; one, two and four
  // through 8192 (16 partials a row) 13.7 and 17.5, 16 and 20, 25 and 28; six to twelve (11 to 6) alike within 0.3; 16 (6)
  // 61 and 59; 12 tokens behind 30000 33 and 68, behind 8192 19 and 22, 16 there 24 and 22; 64 behind 32768 (256 groups) 70 and 53.
  // Deep and many: 64 tokens behind 32768 (256 groups) 53 and 57, 24 sequences of 3 rows behind 8192 (288) 32 and 35, 32 of 5
  // (640) 47.5 and 45.5, 64 of 9 behind 6000 104 and 85, 64 of 25 behind 9000 263 and 201.  Many, blocks over all, 6, 10 or 20
  // an SM: 64 of 9 85, 85 and 87, 64 of 25 202, 202 and 207.
  if (groups <= kMaxBlocks / 2 && parts > 12)
    return launch_after(join_kernel<D, M, KINDS, kSplit>, dim3(all.x, all.y, D / 16), 256, 0, st, p, a);
  if (groups <= 2 * kMaxBlocks) return launch_after(join_kernel<D, M, KINDS, kDeep>, all, 2 * D, 0, st, p, a);
  const int y = std::max(1, std::min((most + 7) / 8, (10 * kMaxBlocks + jobs - 1) / jobs));
  return launch_after(join_kernel<D, M, KINDS, kMany>, dim3(jobs, y), 2 * D, 0, st, p, a);
}

int attend(const mk_cache_shape& c, const SpanCall& call, Params<SpanPlan>& p, const int32_t* block_tables, const void* q,
           int64_t q_stride, const void* kv_layer, void* out, const mk_span_workspace& given, int32_t* status_out,
           mk_stream_t stream) {
  const bool take = given.take != nullptr && call.bytes() > 0;
  int rc = check_attention(c, p.seqs, block_tables, q, q_stride, kv_layer, out, given.ptr, given.bytes, take ? 0 : call.bytes());
  if (rc) return rc;
  const int rows = p.seqs.row0[p.seqs.n];
  void* workspace = take ? given.take(given.ctx, call.bytes()) : given.ptr;
  if (take && !workspace) return chunk_fail(MK_ERR_OOM, "no workspace of %zu bytes", call.bytes());
  if (misaligned(workspace, 16)) return chunk_fail(MK_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  const bool q8 = (c.flags & MK_FLAG_KV_Q8) != 0;
  fill_params(c, block_tables, q, q_stride, kv_layer, out, status_out, &p);
  p.box = span_box(c);
  float* floats = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + call.stage_bytes);
  p.whole = floats + call.whole0;
  const float* part[kRowKinds];
  // Each launch may begin while the kernel before it still runs (launch_after).  The first kernel of the call sets itself
  // up and then waits for that one.  The others need not: none reads what another of them writes, but the staged tiles
  // and the partials, for which their readers wait; and each waits at its end, so that whoever waits for the last one
  // waits for all.
  bool first = true;
  cudaError_t e = cudaSuccess;
  for (int k = 0; k < kRowKinds && e == cudaSuccess; ++k) {
    part[k] = floats + call.part0[k];
    if (call.plan[k].items == 0) continue;
    p.plan = call.plan[k];
    p.first = first && k != kStagedRows;
    p.part = floats + call.part0[k];
    p.folds = call.folds[k] ? floats + call.fold0[k] : nullptr;
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
      e = launch_after(stage_kernel<128, SpanPlan>, dim3(call.stage_tiles, 2 * c.num_kv_heads), kStageThreads, 0, st, p,
                       static_cast<__half*>(workspace), t);
      if (e == cudaSuccess) e = launch<128, kStaged>(p, st);
    } else {
      e = k == kFewRows       ? launch<128, kQ8Few>(p, st)
          : q8                ? launch<128, kQ8>(p, st)
          : c.head_dim == 128 ? launch<128, kBf16>(p, st)
                              : launch<64, kBf16>(p, st);
    }
    first = false;
  }
  if (e == cudaSuccess)
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

extern "C" int mk_window_attention_in(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                      const int32_t* seq_lens, int32_t window, int32_t sinks, const int32_t* block_tables,
                                      const void* q, int64_t q_stride, const void* kv_layer, void* out,
                                      const mk_span_workspace* workspace, int32_t* status_out, mk_stream_t stream) {
  Params<SpanPlan> p;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &p.seqs);
  if (!rc) rc = check_window(window, sinks);
  if (rc) return rc;
  SpanCall call;
  if (!plan_window(*shape, p.seqs, window, sinks, &call)) return too_many();
  return attend(*shape, call, p, block_tables, q, q_stride, kv_layer, out, *workspace, status_out, stream);
}

extern "C" int mk_window_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                   const int32_t* seq_lens, int32_t window, int32_t sinks, const int32_t* block_tables,
                                   const void* q, int64_t q_stride, const void* kv_layer, void* out, void* workspace,
                                   size_t workspace_bytes, int32_t* status_out, mk_stream_t stream) {
  const mk_span_workspace given = {workspace, workspace_bytes, nullptr, nullptr};
  return mk_window_attention_in(shape, num_seqs, chunk_lens, seq_lens, window, sinks, block_tables, q, q_stride, kv_layer, out,
                                &given, status_out, stream);
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

extern "C" int mk_prefix_attention_in(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                      const int32_t* seq_lens, int32_t num_groups, const int32_t* group_seqs,
                                      const int32_t* prefix_lens, const int32_t* block_tables, const void* q, int64_t q_stride,
                                      const void* kv_layer, void* out, const mk_span_workspace* workspace, int32_t* status_out,
                                      mk_stream_t stream) {
  Params<SpanPlan> p;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &p.seqs);
  if (!rc) rc = check_groups(p.seqs, num_groups, group_seqs, prefix_lens);
  if (rc) return rc;
  SpanCall call;
  if (!plan_prefix(*shape, p.seqs, num_groups, group_seqs, prefix_lens, &call)) return too_many();
  return attend(*shape, call, p, block_tables, q, q_stride, kv_layer, out, *workspace, status_out, stream);
}

extern "C" int mk_prefix_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                   const int32_t* seq_lens, int32_t num_groups, const int32_t* group_seqs,
                                   const int32_t* prefix_lens, const int32_t* block_tables, const void* q, int64_t q_stride,
                                   const void* kv_layer, void* out, void* workspace, size_t workspace_bytes,
                                   int32_t* status_out, mk_stream_t stream) {
  const mk_span_workspace given = {workspace, workspace_bytes, nullptr, nullptr};
  return mk_prefix_attention_in(shape, num_seqs, chunk_lens, seq_lens, num_groups, group_seqs, prefix_lens, block_tables, q,
                                q_stride, kv_layer, out, &given, status_out, stream);
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
          int unseen = 0, unseen_n = 0;
          if (k == kStagedRows) unseen_of(pl, g.entry, unseen, unseen_n);
          const int32_t row[21] = {k,     b,       g.entry, g.s,  g.row0,  g.ntok, g.kvh,    g.head,         g.gap,
                                   g.pos0, g.len,  g.tile0, g.pair ? g.n / 2 : g.n,  g.tiles, g.slot, e.stage0, e.stage_tile0, e.stage_head, g.pair,
                                   unseen, unseen_n};
          std::copy(row, row + 21, segments + 21 * static_cast<size_t>(n));
        }
        ++n;
      }
    }
  }
  *n_out = n;
  return MK_OK;
}
