// mk_chunk_attn.cu -- causal attention of a chunk of new tokens over the paged KV cache
// (mk_chunk_attention), on the fifth-generation tensor cores.
//
// out[r][h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(s_t - m),  s_t = q . k_t / sqrt(D),  t <= pos(r)
// in one pass over the positions with a running reference m and sum (exact for any m).
//
// Tiles.  The G query heads of a KV head share its keys, so a tile's 128 rows are TT = 128/G
// tokens times G heads and the causal edge of a tile is TT tokens wide.  A block takes up to two
// tiles of one KV head (a "unit") and streams its positions 128 at a time:
//   S = Q K^T   (128 x 128, K = D)    operands in shared memory, accumulator in tensor memory
//   P = 2^(S c - m c)                  by the tile's warpgroup, a thread per row, bf16 back into
//                                      the columns of S
//   O += P V    (128 x D, K = 128)    P from tensor memory, V from shared memory
// Two tiles in turn keep the tensor cores busy while the other tile's softmax runs: tensor
// memory holds S and O of both (512 columns at D = 128).  A unit with one tile only (a few new
// tokens, as in decoding) runs two STREAMS instead: even and odd position tiles, each with its own
// S, O, m and l, merged at the end.
//
// Roles.  Warps 0-3 and 4-7: softmax and epilogue of tile (stream) 0 and 1.  Warp 8: loads.  Warp
// 9: issues the MMAs.  Over a q8_0 cache warps 12-15 decode codes into the bf16 tiles.  Every
// wait is bounded: one that runs out raises the block's abort flag, every role leaves its loop,
// copies in flight are waited for and tensor memory is returned.
//
// Long contexts with few rows are split over the positions (the host's plan); the partial
// (O, m, l) of each split go to the workspace and a second kernel merges them in split order.

#include "mk_chunk.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

namespace mk {
namespace {

constexpr int kTile = 128;          // positions of a tile, and rows of a tile
constexpr int kRawPos = 64;         // q8_0: positions of one raw stage
constexpr int kRawBytes = kRawPos * (128 + 8);
constexpr int kMasks = 8;           // tiles whose page masks are kept (more than can be in flight)
constexpr uint64_t kWaitNs = 2000000000ull;

// Which work each block takes.  Sequences with rows, longest first; within one, units from the
// last tokens (most positions) to the first, then KV heads, then splits.
struct AttnPlan {
  int32_t n;                        // sequences with rows
  int32_t split_tiles;              // position tiles of a split
  int32_t seq[kMaxSeqs];
  int32_t item0[kMaxSeqs + 1];      // first block of the i-th
  int32_t nsplit[kMaxSeqs];         // by sequence; 1: its blocks write the output
  int64_t part0[kMaxSeqs];          // by sequence: first float of its partials
};

struct AttnParams {
  CUtensorMap map;                  // bf16 pages (see encode_pages)
  ChunkSeqs seqs;
  AttnPlan plan;
  const uint8_t* kv;
  const int32_t* bt;
  int32_t* status;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* part;
  size_t code_bytes;
  int32_t Hq, Hkv, G, TT, ps, P, maxpg;
  int32_t box;                      // positions of one copy: a power of two that divides ps
  float c;                          // log2(e) / sqrt(D)
};

// --------------------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t tx) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(tx) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void tma_5d(uint32_t dst, const void* map, int z, int pg, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(z), "r"(pg), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Shared-memory operand with the 128-byte swizzle: start address; lbo, sbo: bytes between the
// 64-element spans of a row (used where rows run along the operand's K) and between 8-row groups.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 operands, fp32 accumulator; b_mn: B is stored with its N dimension contiguous
__device__ __forceinline__ constexpr uint32_t tc_idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// one elected lane of the converged warp issues
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// columns of this warp's 32 lanes, a lane per thread; not waited for
__device__ __forceinline__ void tc_ld32(uint32_t a, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t a, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t a, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x = *reinterpret_cast<uint64_t*>(&a), y = *reinterpret_cast<uint64_t*>(&b), z = *reinterpret_cast<uint64_t*>(&c), d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x = *reinterpret_cast<uint64_t*>(&a), y = *reinterpret_cast<uint64_t*>(&b), d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t x = *reinterpret_cast<uint64_t*>(&a), y = *reinterpret_cast<uint64_t*>(&b), d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {   // a in the low half
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// --------------------------------------------------------------------------- shared memory
template <int D, bool Q8>
struct Layout {
  static constexpr int kTileBytes = kTile * D * 2;           // one operand tile
  static constexpr int kGroup = D / 64 * 1024;               // 8 positions of a K or V tile
  static constexpr int kQ = 0;                               // two Q tiles
  static constexpr int kRaw = 2 * kTileBytes;                // q8_0: raw stages (a one-tile unit's start at
  static constexpr int kRawStages = Q8 ? 3 : 0;              // the second Q tile)
  static constexpr int kRawStages1 = Q8 ? (kTileBytes + 3 * kRawBytes) / kRawBytes : 0;
  static constexpr int kKv = (kRaw + kRawStages * kRawBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = Q8 ? 4 : D == 128 ? 5 : 8;
  static constexpr int kCtl = kKv + kStages * kTileBytes;
  static constexpr int kThreads = Q8 ? 512 : 384;
};

struct Ctl {
  uint64_t full[8], empty[8];        // K and V tiles: position tile j is ring entries 2j (K) and 2j+1 (V)
  uint64_t raw_full[8], raw_empty[8];
  uint64_t qbar[2], sfull[2], pfull[2], ofull;
  uint32_t tmem, abort;
  uint32_t mask[kMasks];             // per tile, a bit per 8 positions: the page is in range
  float m[kTile], l[kTile];          // stream 1's statistics for the merge
};
static_assert(sizeof(Ctl) <= 2048, "");

template <int D, bool Q8>
constexpr size_t smem_bytes() { return Layout<D, Q8>::kCtl + sizeof(Ctl) + 1024; }
static_assert(smem_bytes<128, false>() <= 232448 && smem_bytes<128, true>() <= 232448 && smem_bytes<64, false>() <= 232448, "");
static_assert(Layout<128, true>::kRawStages1 <= 8, "");

// Waits for the phase of `bar` with this parity, at most kWaitNs; false once the block gives up.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, Ctl* ctl, int32_t* status) {
  volatile uint32_t* abort = &ctl->abort;
  const uint64_t t0 = globaltimer();
  while (!mbar_try(bar, parity)) {
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitNs) {
      *abort = 1u;
      if (status) *status = MK_ERR_TIMEOUT;
      return false;
    }
  }
  return true;
}
// The whole warp waits and agrees on the outcome (and is converged for what follows).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, Ctl* ctl, int32_t* status) {
  return __all_sync(~0u, mbar_try(bar, parity) || mbar_wait_slow(bar, parity, ctl, status));
}

// What one block does.
struct Item {
  int s, kvh, split, nsplit;
  int tok0, ntok;        // tokens of the unit within the sequence's new ones
  int pos0;              // position of the unit's first token
  int len;
  int tile0, n;          // position tiles [tile0, tile0 + n)
  bool two;              // two Q tiles (else two streams of one)
};

__device__ __forceinline__ bool find_item(const AttnParams& p, Item& it) {
  const int b = blockIdx.x;
  int lo = 0, hi = p.plan.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.plan.item0[mid] <= b) lo = mid;
    else hi = mid;
  }
  it.s = p.plan.seq[lo];
  it.nsplit = p.plan.nsplit[it.s];
  it.len = p.seqs.len[it.s];
  const int chunk = p.seqs.row0[it.s + 1] - p.seqs.row0[it.s];
  const int UT = 2 * p.TT, nu = (chunk + UT - 1) / UT;
  int rem = b - p.plan.item0[lo];
  const int u = nu - 1 - rem / (p.Hkv * it.nsplit);
  rem %= p.Hkv * it.nsplit;
  it.kvh = rem / it.nsplit;
  it.split = rem % it.nsplit;
  it.tok0 = u * UT;
  it.ntok = min(UT, chunk - it.tok0);
  it.pos0 = it.len - chunk + it.tok0;
  it.two = it.ntok > p.TT;
  const int tiles = (it.pos0 + it.ntok - 1) / kTile + 1;
  it.tile0 = it.split * p.plan.split_tiles;
  it.n = it.nsplit == 1 ? tiles : min(p.plan.split_tiles, tiles - it.tile0);
  return it.n > 0;       // (an early unit has fewer tiles than the sequence's last)
}

// First float of the partials of (unit u, KV head, split) of a sequence: rows of D + 4 floats
// (O, then m, l), `urows` of them per split.
__device__ __forceinline__ size_t part_at(const AttnParams& p, int s, int u, int kvh, int split, int D) {
  const int chunk = p.seqs.row0[s + 1] - p.seqs.row0[s];
  const int urows = min(chunk, 2 * p.TT) * p.G;
  return p.plan.part0[s] +
         (static_cast<size_t>(u * p.Hkv + kvh) * p.plan.nsplit[s] + split) * urows * static_cast<size_t>(D + 4);
}

// --------------------------------------------------------------------------- loads (warp 8)
template <int D, bool Q8>
__device__ __forceinline__ void produce(const AttnParams& p, const Item& it, uint32_t base, Ctl* ctl) {
  using L = Layout<D, Q8>;
  const int lane = threadIdx.x & 31;
  const int r = p.box, nbox = (Q8 ? kRawPos : kTile) / r;     // copies of a stage
  const int32_t* bt = p.bt + static_cast<size_t>(it.s) * p.maxpg;
  // lane b looks up the page of the tile's b-th copy, one tile ahead
  constexpr int kPerTile = Q8 ? 2 : 1;
  auto lookup = [&](int j) {
    const int pos = (it.tile0 + j) * kTile + lane * r;
    return j < it.n && lane < nbox * kPerTile && pos < it.len ? __ldg(bt + pos / p.ps) : -1;
  };
  const uint32_t raw0 = base + (it.two ? L::kRaw : L::kTileBytes);
  const int nraw = it.two ? L::kRawStages : L::kRawStages1;
  int page_next = lookup(0);
  int u = 0;                                                   // q8_0: raw stages filled
  for (int j = 0; j < it.n; ++j) {
    const int page = page_next;
    page_next = lookup(j + 1);
    const int pos = (it.tile0 + j) * kTile + lane * r;
    const bool mine = lane < nbox * kPerTile;
    const bool good = page >= 0 && page < p.P;
    if (mine && pos < it.len && !good && p.status) *p.status = MK_ERR_DEVICE_BOUNDS;
    const int off = pos % p.ps;
    // a bit per 8 positions
    const uint32_t ok = __ballot_sync(~0u, mine && good);
    const uint32_t mask = __ballot_sync(~0u, lane < 16 && ((ok >> (lane * 8 / r)) & 1u));
    if (lane == 0) ctl->mask[j % kMasks] = mask;
    if constexpr (!Q8) {
      for (int which = 0; which < 2; ++which) {
        const int c = 2 * j + which, st = c % L::kStages;
        const uint32_t bar = smem_u32(&ctl->full[st]);
        if (!mbar_wait(smem_u32(&ctl->empty[st]), ((c / L::kStages) & 1) ^ 1, ctl, p.status)) return;
        if (lane == 0) mbar_expect(bar, L::kTileBytes);
        __syncwarp();
        // a copy out of the pool's range fills its positions with zeros
        if (mine)
          tma_5d(base + L::kKv + st * L::kTileBytes + lane * (r / 8) * L::kGroup, &p.map, (it.kvh * p.ps + off) / 8,
                 (good ? page : p.P) * 2 + which, bar);
      }
    } else {
      for (int which = 0; which < 2; ++which)
        for (int h = 0; h < 2; ++h, ++u) {
          const int st = u % nraw;
          const uint32_t bar = smem_u32(&ctl->raw_full[st]), dst = raw0 + st * kRawBytes;
          if (!mbar_wait(smem_u32(&ctl->raw_empty[st]), ((u / nraw) & 1) ^ 1, ctl, p.status)) return;
          const bool copy = mine && good && lane / nbox == h;
          const int cnt = __popc(__ballot_sync(~0u, copy));
          if (lane == 0) mbar_expect(bar, cnt * r * 136);
          __syncwarp();
          if (copy) {
            const size_t line = (static_cast<size_t>(page) * 2 + which) * p.Hkv * p.ps +
                                static_cast<size_t>(it.kvh) * p.ps + off;
            const int b = lane - h * nbox;
            bulk_g2s(dst + b * r * 128, p.kv + line * 128, r * 128, bar);
            bulk_g2s(dst + kRawPos * 128 + b * r * 8, p.kv + p.code_bytes + line * 8, r * 8, bar);
          }
        }
    }
  }
}

// --------------------------------------------------------------------------- q8_0 (warps 12-15)
// Codes to bf16 tiles in the operand layout.  A code becomes fp32 exactly (its byte with the sign
// flipped is the low mantissa byte of 2^23 + 128 + code), times its f16 scale in fp32, rounded
// once to bf16.  Positions of pages out of range or behind the sequence become zeros.
template <int D>
__device__ __forceinline__ void decode(const AttnParams& p, const Item& it, uint32_t base, Ctl* ctl) {
  using L = Layout<D, true>;
  const int tid = threadIdx.x & 127;
  const uint32_t raw0 = base + (it.two ? L::kRaw : L::kTileBytes);
  const int nraw = it.two ? L::kRawStages : L::kRawStages1;
  const int piece = tid & 7, row0 = tid >> 3;       // 16 codes of rows row0 + 16 i
  int u = 0;
  for (int j = 0; j < it.n; ++j) {
    const int p0 = (it.tile0 + j) * kTile;
    for (int which = 0; which < 2; ++which) {
      const int c = 2 * j + which, st = c % L::kStages;
      if (!mbar_wait(smem_u32(&ctl->empty[st]), ((c / L::kStages) & 1) ^ 1, ctl, p.status)) return;
      const uint32_t dst = base + L::kKv + st * L::kTileBytes + (piece >> 2) * 1024;
      for (int h = 0; h < 2; ++h, ++u) {
        const int rs = u % nraw;
        const uint32_t src = raw0 + rs * kRawBytes;
        if (!mbar_wait(smem_u32(&ctl->raw_full[rs]), (u / nraw) & 1, ctl, p.status)) return;
        const uint32_t mask = ctl->mask[j % kMasks];
#pragma unroll
        for (int i = 0; i < kRawPos / 16; ++i) {
          const int row = row0 + 16 * i, n = h * kRawPos + row;
          uint32_t w[4];
          uint16_t sc;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(src + row * 128 + piece * 16));
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sc) : "r"(src + kRawPos * 128 + row * 8 + (piece >> 1) * 2));
          const float d = __half2float(__ushort_as_half(sc));
          const bool live = ((mask >> (n >> 3)) & 1u) && p0 + n < it.len;
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t x = w[k] ^ 0x80808080u;
            float2 a, b;
            a.x = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7440));
            a.y = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7441));
            b.x = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7442));
            b.y = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7443));
            const float2 off = make_float2(-8388736.f, -8388736.f), dd = make_float2(d, d);
            a = mul2(add2(a, off), dd);
            b = mul2(add2(b, off), dd);
            o[2 * k] = live ? bf16x2(a.x, a.y) : 0u;
            o[2 * k + 1] = live ? bf16x2(b.x, b.y) : 0u;
          }
          const uint32_t at = dst + (n >> 3) * L::kGroup + (n & 7) * 128;
          const uint32_t ch = (piece & 3) * 2;
          sts16(at + ((ch ^ (n & 7)) << 4), o[0], o[1], o[2], o[3]);
          sts16(at + (((ch + 1) ^ (n & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(smem_u32(&ctl->raw_empty[rs]));
      }
      fence_async_smem();
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(smem_u32(&ctl->full[st]));
    }
  }
}

// --------------------------------------------------------------------------- MMAs (warp 9)
template <int D, bool Q8>
__device__ __forceinline__ void issue(const AttnParams& p, const Item& it, uint32_t base, Ctl* ctl, uint32_t tm) {
  using L = Layout<D, Q8>;
  constexpr uint32_t kIdS = tc_idesc(kTile, kTile, false), kIdO = tc_idesc(kTile, D, true);
  const int lane = threadIdx.x & 31;
  auto ring = [&](int c) { return c % L::kStages; };
  auto wait_full = [&](int c) {
    const bool ok = mbar_wait(smem_u32(&ctl->full[ring(c)]), (c / L::kStages) & 1, ctl, p.status);
    tc_after();
    return ok;
  };
  auto release = [&](int c) { tc_commit(smem_u32(&ctl->empty[ring(c)])); };
  auto scores = [&](int t, int qt, int j) {        // S of tile (stream) t from Q tile qt and K tile j
    const uint64_t a = tc_desc(base + qt * L::kTileBytes, 16, 1024);
    const uint64_t b = tc_desc(base + L::kKv + ring(2 * j) * L::kTileBytes, 16, L::kGroup);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      mma_ss(tm + t * kTile, a + (k / 4) * (kTile * 128 >> 4) + (k % 4) * 2, b + (k / 4) * (1024 >> 4) + (k % 4) * 2, kIdS,
             k > 0);
    tc_commit(smem_u32(&ctl->sfull[t]));
    // the page mask travels with an ordinary arrival: the warp that wrote it arrived on `full`
    if (lane == 0) mbar_arrive(smem_u32(&ctl->sfull[t]));
  };
  auto values = [&](int t, int j, bool acc) {      // O of tile (stream) t += P V tile j
    const uint64_t b = tc_desc(base + L::kKv + ring(2 * j + 1) * L::kTileBytes, 1024, L::kGroup);
#pragma unroll
    for (int k = 0; k < kTile / 16; ++k)
      mma_ts(tm + 2 * kTile + t * D, tm + t * kTile + k * 8, b + k * (2 * L::kGroup >> 4), kIdO, acc || k > 0);
  };
  // bf16: what a page holds behind the sequence's last position must not meet a weight, not even
  // a zero one (0 * NaN): zeros instead.  (q8_0 tiles are zeroed as they are decoded.)
  auto trim = [&](int j) {
    const int first = it.len - (it.tile0 + j) * kTile;
    if (Q8 || first >= kTile) return;
    const int last = (first + p.box - 1) / p.box * p.box;      // copies behind are zeros already
    const uint32_t v = base + L::kKv + ring(2 * j + 1) * L::kTileBytes;
    for (int n = first; n < last; ++n)
      if (lane < D / 8) sts16(v + (n >> 3) * L::kGroup + (lane >> 3) * 1024 + (n & 7) * 128 + (lane & 7) * 16, 0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
  };
  auto wait_p = [&](int t, int i) {
    const bool ok = mbar_wait(smem_u32(&ctl->pfull[t]), i & 1, ctl, p.status);
    tc_after();
    return ok;
  };
  if (!mbar_wait(smem_u32(&ctl->qbar[0]), 0, ctl, p.status)) return;
  if (it.two) {
    if (!mbar_wait(smem_u32(&ctl->qbar[1]), 0, ctl, p.status)) return;
    tc_after();
    if (!wait_full(0)) return;
    scores(0, 0, 0);
    scores(1, 1, 0);
    release(0);
    for (int j = 0; j < it.n; ++j) {
      const bool more = j + 1 < it.n;
      if (!wait_p(0, j) || !wait_full(2 * j + 1)) return;
      trim(j);
      values(0, j, j > 0);
      if (more) {
        if (!wait_full(2 * j + 2)) return;
        scores(0, 0, j + 1);
      }
      if (!wait_p(1, j)) return;
      values(1, j, j > 0);
      release(2 * j + 1);
      if (more) {
        scores(1, 1, j + 1);
        release(2 * j + 2);
      }
    }
  } else {
    tc_after();
    for (int j = 0; j < 2 && j < it.n; ++j) {
      if (!wait_full(2 * j)) return;
      scores(j, 0, j);
      release(2 * j);
    }
    for (int j = 0; j < it.n; ++j) {
      const int t = j & 1;
      if (!wait_p(t, j >> 1) || !wait_full(2 * j + 1)) return;
      trim(j);
      values(t, j, j > 1);
      release(2 * j + 1);
      if (j + 2 < it.n) {
        if (!wait_full(2 * j + 4)) return;
        scores(t, 0, j + 2);
        release(2 * j + 4);
      }
    }
  }
  tc_commit(smem_u32(&ctl->ofull));
}

// --------------------------------------------------------------------------- softmax (warps 0-7)
template <int D, bool Q8>
__device__ __forceinline__ void softmax(const AttnParams& p, const Item& it, uint32_t base, uint8_t* smem, Ctl* ctl,
                                        uint32_t tm) {
  using L = Layout<D, Q8>;
  const int t = threadIdx.x >> 7, row = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int urow0 = it.two ? t * p.TT * p.G : 0;    // first row of the tile within the unit
  const int trows = p.TT * p.G;
  const int rows = min(trows, it.ntok * p.G - urow0);
  // the tile's query rows into the operand layout (K-major, 128-byte swizzle), zeros behind them
  if (it.two || t == 0) {
    const uint16_t* q = p.q + static_cast<size_t>(p.seqs.row0[it.s] + it.tok0 + (it.two ? t * p.TT : 0)) * p.q_stride +
                        static_cast<size_t>(it.kvh) * p.G * D;
    const uint32_t dst = base + t * L::kTileBytes;
    constexpr int CH = D / 8;
#pragma unroll 8
    for (int i = 0; i < CH; ++i) {
      const int x = i * 128 + row, rr = x / CH, ch = x % CH;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (rr < rows) {
        const int tok = rr / p.G;
        w = __ldg(reinterpret_cast<const uint4*>(q + tok * p.q_stride + (rr - tok * p.G) * D) + ch);
      }
      sts16(dst + (ch >> 3) * (kTile * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), w.x, w.y, w.z, w.w);
    }
    fence_async_smem();
    mbar_arrive(smem_u32(&ctl->qbar[t]));
  }
  const bool live = row < rows;
  // rows behind the last see everything, so that they never ask for a mask
  const int pos = live ? it.pos0 + (it.two ? t * p.TT : 0) + row / p.G : INT32_MAX;
  const int mine = it.two ? it.n : (it.n - t + 1) / 2;
  const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t ts = tm + t * kTile + lane_base, to = tm + 2 * kTile + t * D + lane_base;
  const float c = p.c, grow = 8.0f / c;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int i = 0; i < mine; ++i) {
    const int j = it.two ? i : 2 * i + t;
    ok = mbar_wait(smem_u32(&ctl->sfull[t]), i & 1, ctl, p.status);
    if (!ok) break;
    tc_after();
    float s[kTile];
#pragma unroll
    for (int k = 0; k < kTile; k += 32) tc_ld32(ts + k, s + k);
    tc_wait_ld();
    const int limit = pos - (it.tile0 + j) * kTile;          // last column this row sees
    const uint32_t mask = ctl->mask[j % kMasks];
    if (__any_sync(~0u, limit < kTile - 1 || mask != 0xffffu)) {
#pragma unroll
      for (int k = 0; k < kTile; ++k)
        if (k > limit || !((mask >> (k >> 3)) & 1u)) s[k] = -INFINITY;
    }
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < kTile; ++k) mx[k % 4] = fmaxf(mx[k % 4], s[k]);
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    // The reference moves only when the maximum outgrows it by 2^8: until then weights up to 2^8
    // are as exact in bf16 and fp32 as weights up to 1, and O needs no rescaling.
    if (i == 0) {
      m = top;
    } else {
      const bool up = top > m + grow;
      if (__any_sync(~0u, up)) {
        const float mn = up ? top : m;
        const float f = m == -INFINITY ? 0.f : ex2((m - mn) * c);
        l *= f;
        m = mn;
        // the previous P V is complete: S, issued after it, is
        const float2 ff = make_float2(f, f);
#pragma unroll
        for (int k = 0; k < D; k += 16) {
          float o[16];
          tc_ld16(to + k, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 x = mul2(make_float2(o[e], o[e + 1]), ff);
            o[e] = x.x;
            o[e + 1] = x.y;
          }
          tc_st16(to + k, o);
        }
      }
    }
    const float mb = m == -INFINITY ? 0.f : -m * c;
    const float2 cc = make_float2(c, c), mm = make_float2(mb, mb);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int e = h * 32 + 2 * k;
        const float2 x = fma2(make_float2(s[e], s[e + 1]), cc, mm);
        const float2 y = make_float2(ex2(x.x), ex2(x.y));
        sum[k & 1] = add2(sum[k & 1], y);
        w[k] = bf16x2(y.x, y.y);
      }
      tc_st16(ts + h * 16, w);
    }
    const float2 sm = add2(sum[0], sum[1]);
    l += sm.x + sm.y;
    tc_wait_st();
    tc_before();
    mbar_arrive(smem_u32(&ctl->pfull[t]));
  }
  if (ok) ok = mbar_wait(smem_u32(&ctl->ofull), 0, ctl, p.status);
  tc_after();
  // m and l in powers of two; a row without a position has m = -inf and l = 0
  m = m == -INFINITY ? m : m * c;
  float f0 = 1.f, f1 = 0.f;
  float* other = reinterpret_cast<float*>(smem + L::kQ);   // stream 1's O, [D][128]: every MMA has read Q by now
  const bool merge = !it.two;
  if (merge) {
    if (t == 1 && ok && warp * 32 < rows) {
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        if (mine > 0) {
          tc_ld32(to + k, o);
          tc_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) other[(k + e) * 128 + row] = mine > 0 ? o[e] : 0.f;
      }
      ctl->m[row] = m;
      ctl->l[row] = l;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (t == 1) return;
    const float m1 = ctl->m[row], l1 = ctl->l[row];
    const float mt = fmaxf(m, m1);
    if (mt != -INFINITY) {
      f0 = ex2(m - mt);
      f1 = ex2(m1 - mt);
    }
    l = l * f0 + l1 * f1;
    m = mt;
  }
  if (!ok || warp * 32 >= rows) return;
  const int urow = urow0 + row, tok = it.tok0 + urow / p.G, g = urow % p.G;
  float* part = nullptr;
  uint16_t* out = nullptr;
  float inv = 1.f;
  if (it.nsplit > 1) {
    part = p.part + part_at(p, it.s, it.tok0 / (2 * p.TT), it.kvh, it.split, D) + static_cast<size_t>(urow) * (D + 4);
  } else {
    out = p.out + (static_cast<size_t>(p.seqs.row0[it.s] + tok) * p.Hq + it.kvh * p.G + g) * D;
    inv = l == 0.f ? 0.f : 1.0f / l;
  }
#pragma unroll 1
  for (int k = 0; k < D; k += 32) {
    float x[32];
    tc_ld32(to + k, x);
    tc_wait_ld();
    if (merge) {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = x[e] * f0 + other[(k + e) * 128 + row] * f1;
    }
    if (live && part != nullptr) {
#pragma unroll
      for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(part + k + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else if (live) {
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint4 w;
        w.x = bf16x2(x[e] * inv, x[e + 1] * inv);
        w.y = bf16x2(x[e + 2] * inv, x[e + 3] * inv);
        w.z = bf16x2(x[e + 4] * inv, x[e + 5] * inv);
        w.w = bf16x2(x[e + 6] * inv, x[e + 7] * inv);
        *reinterpret_cast<uint4*>(out + k + e) = w;
      }
    }
    __syncwarp();
  }
  if (part != nullptr && live) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
}

template <int D, bool Q8>
__global__ void __launch_bounds__(Layout<D, Q8>::kThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<D, Q8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + L::kCtl);
  const int warp = threadIdx.x >> 5;
  Item it;
  if (!find_item(p, it)) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), Q8 ? 4 : 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
      mbar_init(smem_u32(&ctl->raw_full[i]), 1);
      mbar_init(smem_u32(&ctl->raw_empty[i]), 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ctl->qbar[t]), 128);
      mbar_init(smem_u32(&ctl->sfull[t]), 2);
      mbar_init(smem_u32(&ctl->pfull[t]), 128);
    }
    mbar_init(smem_u32(&ctl->ofull), 1);
    ctl->abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = ctl->tmem;
  // registers follow the work: a softmax thread holds a row of S (sum over the warpgroups within the launch's)
  if (warp < 8) {
    if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    softmax<D, Q8>(p, it, base, smem, ctl, tm);
  } else if (warp < 12) {
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) produce<D, Q8>(p, it, base, ctl);
    if (warp == 9) issue<D, Q8>(p, it, base, ctl, tm);
  } else if constexpr (Q8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    decode<D>(p, it, base, ctl);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (ctl->abort) {
    // an aborted block may leave copies and MMAs in flight: they must end before its shared and
    // tensor memory are another block's
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 100000000ull) __nanosleep(1000000);
    __syncthreads();
  }
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
}

// Merges the splits of split sequences, in split order: a warp per (row, query head).
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ AttnParams p) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= static_cast<int64_t>(p.seqs.row0[p.seqs.n]) * p.Hq) return;
  const int r = static_cast<int>(unit / p.Hq), h = static_cast<int>(unit - static_cast<int64_t>(r) * p.Hq);
  const int s = seq_of_row(p.seqs, r), ns = p.plan.nsplit[s];
  if (ns == 1) return;
  const int chunk = p.seqs.row0[s + 1] - p.seqs.row0[s], i = r - p.seqs.row0[s], UT = 2 * p.TT, u = i / UT;
  const int last = p.seqs.len[s] - chunk + min(chunk, (u + 1) * UT) - 1;       // the unit's last position
  const int n = (last / kTile) / p.plan.split_tiles + 1;                       // splits it has
  const int urows = min(chunk, UT) * p.G, urow = (i - u * UT) * p.G + h % p.G;
  const float* part = p.part + part_at(p, s, u, h / p.G, 0, D) + static_cast<size_t>(urow) * (D + 4);
  const size_t step = static_cast<size_t>(urows) * (D + 4);
  float M = -INFINITY;
  for (int k = lane; k < n; k += 32) M = fmaxf(M, part[k * step + D]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
  constexpr int V = D / 32;
  float acc[V] = {}, L = 0.f;
  if (M != -INFINITY)
    for (int k = 0; k < n; ++k) {
      const float* pk = part + k * step;
      const float2 ml = *reinterpret_cast<const float2*>(pk + D);
      const float f = ex2(ml.x - M);
      L += f * ml.y;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(f, pk[lane * V + v], acc[v]);
    }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  uint16_t* out = p.out + (static_cast<size_t>(r) * p.Hq + h) * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(out + v) = bf16x2(acc[v] * inv, acc[v + 1] * inv);
}

// --------------------------------------------------------------------------- host
constexpr int kSms = 152;

// Splits the positions so that the blocks come out even, where they would not by themselves.
// Returns the number of blocks; *floats: the workspace.
int64_t make_plan(const mk_cache_shape& c, const ChunkSeqs& q, AttnPlan* pl, size_t* floats) {
  const int G = c.num_q_heads / c.num_kv_heads, UT = 2 * (kTile / G);
  pl->n = 0;
  int64_t work = 0;
  for (int s = 0; s < q.n; ++s) {
    const int chunk = q.row0[s + 1] - q.row0[s];
    pl->nsplit[s] = 1;
    pl->part0[s] = 0;
    if (chunk == 0) continue;
    pl->seq[pl->n++] = s;
    for (int64_t t0 = 0; t0 < chunk; t0 += UT)
      work += int64_t(c.num_kv_heads) * ((q.len[s] - chunk + std::min<int64_t>(chunk, t0 + UT) - 1) / kTile + 1);
  }
  std::sort(pl->seq, pl->seq + pl->n, [&](int a, int b) { return q.len[a] != q.len[b] ? q.len[a] > q.len[b] : a < b; });
  const int64_t even = (work + kSms - 1) / kSms;
  pl->split_tiles = static_cast<int32_t>(std::max<int64_t>(even, 4));
  int64_t items = 0;
  size_t at = 0;
  for (int i = 0; i < pl->n; ++i) {
    const int s = pl->seq[i], chunk = q.row0[s + 1] - q.row0[s];
    const int64_t units = (chunk + UT - 1) / UT, tiles = (q.len[s] - 1) / kTile + 1;
    const int64_t ns = (tiles + pl->split_tiles - 1) / pl->split_tiles;
    pl->nsplit[s] = static_cast<int32_t>(ns);
    pl->item0[i] = static_cast<int32_t>(items);
    items += units * c.num_kv_heads * ns;
    if (ns > 1) {
      pl->part0[s] = static_cast<int64_t>(at);
      at += static_cast<size_t>(units * c.num_kv_heads * ns) * std::min(chunk, UT) * G * (c.head_dim + 4);
    }
  }
  pl->item0[pl->n] = static_cast<int32_t>(items);
  *floats = at;
  return items;
}

// bf16 pages to TMA, innermost first: {64 dims, 8 positions, D/64 spans of dims, groups of 8
// positions over the KV heads, pages x (K, V)}.  A box lands as [group][span][8 positions][128 B]:
// 8-position groups a constant distance apart whatever the page size, which is what the operand
// descriptors of both K (rows along dims) and V (rows along positions) need.
int encode_pages(const mk_cache_shape& c, const void* kv, int box_pos, CUtensorMap* out) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)
                                                                : nullptr;
  }();
  if (!encode) return chunk_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t D = c.head_dim, ps = c.page_size, hkv = c.num_kv_heads;
  const cuuint64_t dims[5] = {64, 8, D / 64, hkv * ps / 8, static_cast<cuuint64_t>(c.num_pages) * 2};
  const cuuint64_t strides[4] = {D * 2, 128, 8 * D * 2, hkv * ps * D * 2};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(box_pos / 8), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(kv), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MK_OK : chunk_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
}

template <int D, bool Q8>
cudaError_t launch(const AttnParams& p, unsigned blocks, bool merge, cudaStream_t st) {
  // (idempotent and cheap next to a launch; per device, so set on every call)
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem_bytes<D, Q8>()));
  if (e != cudaSuccess) return e;
  attn_kernel<D, Q8><<<blocks, Layout<D, Q8>::kThreads, smem_bytes<D, Q8>(), st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !merge) return e;
  const int64_t warps = static_cast<int64_t>(p.seqs.row0[p.seqs.n]) * p.Hq;
  merge_kernel<D><<<static_cast<unsigned>((warps + 7) / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
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
  AttnPlan plan;
  size_t floats = 0;
  make_plan(*shape, seqs, &plan, &floats);
  *bytes_out = floats * sizeof(float);
  return MK_OK;
}

extern "C" int mk_chunk_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                  const int32_t* seq_lens, const int32_t* block_tables, const void* q,
                                  int64_t q_stride, const void* kv_layer, void* out, void* workspace,
                                  size_t workspace_bytes, int32_t* status_out, mk_stream_t stream) {
  AttnParams p;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &p.seqs);
  if (rc) return rc;
  const mk_cache_shape& c = *shape;
  if (q_stride < static_cast<int64_t>(c.num_q_heads) * c.head_dim || q_stride % 8)
    return chunk_fail(MK_ERR_INVALID_ARG, "q_stride must be a multiple of 8, at least num_q_heads*head_dim");
  const int rows = p.seqs.row0[num_seqs];
  if (rows > 0 && (!block_tables || !q || !kv_layer || !out))
    return chunk_fail(MK_ERR_INVALID_ARG, "a pointer argument is NULL");
  if (misaligned(block_tables, 4) || misaligned(q, 16) || misaligned(kv_layer, 16) || misaligned(out, 16) ||
      misaligned(workspace, 16))
    return chunk_fail(MK_ERR_INVALID_ARG, "pointers must be 16-byte aligned (block_tables 4-byte)");
  size_t floats = 0;
  const int64_t items = make_plan(c, p.seqs, &p.plan, &floats);
  if (items >= (int64_t(1) << 31)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  if (workspace_bytes < floats * sizeof(float) || (floats > 0 && !workspace))
    return chunk_fail(MK_ERR_INVALID_ARG, "the workspace holds %zu bytes; these lengths need %zu", workspace_bytes,
                      floats * sizeof(float));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  const bool q8 = (c.flags & MK_FLAG_KV_Q8) != 0;
  p.box = std::min(c.page_size & -c.page_size, q8 ? kRawPos : kTile);
  if (!q8) {
    rc = encode_pages(c, kv_layer, p.box, &p.map);
    if (rc) return rc;
  }
  p.kv = static_cast<const uint8_t*>(kv_layer);
  p.bt = block_tables;
  p.status = status_out;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.part = static_cast<float*>(workspace);
  p.code_bytes = static_cast<size_t>(c.num_pages) * 2 * c.num_kv_heads * c.page_size * c.head_dim;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.G = c.num_q_heads / c.num_kv_heads;
  p.TT = kTile / p.G;
  p.ps = c.page_size;
  p.P = c.num_pages;
  p.maxpg = c.max_pages_per_seq;
  p.c = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(c.head_dim)));
  const unsigned blocks = static_cast<unsigned>(items);
  const cudaError_t e = q8 ? launch<128, true>(p, blocks, floats > 0, st)
                           : c.head_dim == 128 ? launch<128, false>(p, blocks, floats > 0, st)
                                               : launch<64, false>(p, blocks, floats > 0, st);
  return e == cudaSuccess ? MK_OK : chunk_fail(MK_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
}
