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
// S, O, m and l, joined at the end.
//
// Roles.  Warps 0-3 and 4-7: softmax and epilogue of tile (stream) 0 and 1.  Warps 8 and 11: K and V
// loads.  Warp 9: issues the MMAs.  Warp 10: query rows and V tails.  Over a q8_0 cache warps 12-15
// decode codes into fp16 operand tiles (units of at most 32 rows: two groups, warps 12-15 K and 16-19 V);
// sequences whose tiles many blocks would decode are decoded once before (stage_kernel).  Blocks are persistent (mk_chunk_plan.h): loads and scores of the next segment
// run under the epilogue of this one.  Every wait is bounded: one that runs out raises the block's abort
// flag, every role leaves its loop, copies in flight are let land and tensor memory is returned.
//
// What bounds it.  Units of two tiles: 4 * 128^3 multiply-adds a position tile need 2048 tensor-core
// cycles and as many of shared memory (192 KB of operands read, 64 KB written, at 128 B a cycle); about
// 2800 are measured (8192-token prompt, 32 heads of 128: 342 us, 1.61 PFLOP/s; the last 2048 of
// 32768 tokens: 635 us, 1.68).  Units of one tile: HBM, 160 KB of copies in flight a block (one token, 131072
// positions: 49.5 us, 5.4 TB/s).  Few rows over a q8_0 cache: the decode, whose two products and byte
// permute per two codes take the half-precision pipe as long as the copies take HBM (one token, 262144
// positions: 71.9 us; without the two products 61, without any work 56).
//
// Operands.  bf16 cache: Q, K, V as they are, P rounded to bf16 (2^-8; its sum uses the unrounded
// values).  q8_0 cache: fp16, whose 2^-11 keeps a decoded value three bits better than bf16 would
// and whose decode is one byte permute, one subtract and one multiply per two codes: K and V are
// code * scale; a row of Q is divided by a power of two (undone in the softmax's constant), so that
// it fits; P carries a factor 2^6, so that small weights stay clear of fp16's subnormals.
//
// What a row does not see must not reach it, and what fp16 cannot hold must still come out right: a row
// whose result is not finite, or whose weights are all zeros, is computed again from the cache in fp32,
// position by position (exact_row).  A NaN or infinity among later V rows of the same tile (0 * NaN) and scales whose values
// overflow fp16 (the decode makes them NaN) end there; a row that really holds a NaN stays one.  A warp takes a
// row and head at a time there: an 8192-token prompt of 32 heads takes 0.36 ms, 1.2 with a NaN in its second key,
// 172 with one in its middle key, 292 with one in an early value (whose other dims go on to the end).

#include "mk_chunk_plan.h"
#include "mk_debug.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

namespace mk {
namespace {

// What the K and V operands come from: bf16 pages; q8_0 pages, decoded by the block; q8_0 pages that a
// kernel before this one has decoded into the workspace (see stage_kernel); q8_0 pages where every unit has
// at most kFew rows (see softmax_few).
enum { kBf16, kQ8, kStaged, kQ8Few };
template <int M>
constexpr bool kDecodes = M == kQ8 || M == kQ8Few;
constexpr int kFew = 32;
constexpr int kRawFew = 2;                     // raw stages of K and of V there

constexpr int kRawBytes = kTile * (128 + 8);   // q8_0: the codes and scales of a K or V tile
constexpr int kMasks = 8;           // tiles whose page masks are kept (more than can be in flight)
constexpr uint64_t kWaitNs = 2000000000ull;

// The staged sequences and their tiles' numbers.
struct StageTiles {
  int32_t n;
  int32_t seq[kMaxSeqs], first[kMaxSeqs + 1];
};

struct AttnParams {
  CUtensorMap map;                  // bf16 pages (see encode_pages)
  CUtensorMap qmap;                 // query rows (see encode_queries)
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
  int32_t stage0[kMaxSeqs];         // staged sequences: first tile in the workspace
  int32_t Hq, ps, P, maxpg;
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
__device__ __forceinline__ void tma_4d(uint32_t dst, const void* map, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(w), "r"(bar)
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
// Shared-memory operand with the 128-byte swizzle, in two words: start address and lbo (bytes between
// the 64-element spans of a row, used where rows run along the operand's K); sbo, bytes between
// 8-row groups, and the constant fields.  Addresses advance in the low word alone.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16; }
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t sbo) { return sbo >> 4 | 1u << 14 | 2u << 29; }
// bf16 (or fp16) operands, fp32 accumulator; b_mn: B is stored with its N dimension contiguous
__device__ __forceinline__ constexpr uint32_t tc_idesc(bool bf16, int M, int N, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// One elected lane of the converged warp issues; the whole warp computes the operands, so that they
// stay in uniform registers (issued from one thread's branch, an 8192-token prompt took 455 us
// instead of 390: every operand moved across for every product).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t ahi, uint32_t b, uint32_t bhi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(ahi), "r"(b), "r"(bhi), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t bhi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(bhi), "r"(idesc), "r"(static_cast<uint32_t>(acc))
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// --------------------------------------------------------------------------- shared memory
template <int D, int M>
struct Layout {
  static constexpr int kTileBytes = kTile * D * 2;           // one operand tile
  static constexpr int kGroup = D / 64 * 1024;               // 8 positions of a K or V tile
  static constexpr int kRawStages = M == kQ8Few ? 2 * kRawFew : 3;
  static constexpr int kRaw = (M == kQ8Few ? 1 : 2) * kTileBytes;   // behind the Q tiles
  static constexpr int kKv = (kRaw + (kDecodes<M> ? kRawStages * kRawBytes : 0) + 1023) / 1024 * 1024;
  static constexpr int kStages = kDecodes<M> ? 3 : D == 128 ? 5 : 8;
  static constexpr int kCtl = kKv + kStages * kTileBytes;
  static constexpr int kThreads = M == kQ8Few ? 640 : M == kQ8 ? 512 : 384;
};

struct Ctl {
  uint64_t full[8], empty[8];        // K and V tiles, a ring (see entry_of)
  uint64_t raw_full[8], raw_empty[8];
  uint64_t qraw[2], qbar[2], qfree;  // query tiles: landed, in the operand type (bf16: qraw itself), read by the last S
  uint64_t sfull[2], pfull[2][2];    // S of a tile (stream); the halves of its P
  uint64_t landed, trim;             // a last V tile to be trimmed: landed, trimmed
  uint64_t ofull, join;
  uint32_t tmem, abort;
  uint32_t beat;                     // counts while a softmax warp works a row out plainly (exact_row)
  uint32_t mask[kMasks];             // per tile, a bit per 8 positions: the page is in range
  float2 ml[2][kTile];               // streams' (m, l) when they join
};
struct CtlQ8 : Ctl {
  float rowc[kTile];                 // two streams: the softmax's constant of each query row
};
struct CtlFew : CtlQ8 {
  uint32_t raw_mask[2 * kRawFew];    // the page mask of a raw stage's tile
  uint64_t shared[2];                // a warpgroup's parts of the output: written, read
  float part[2][16][4][kFew];        // 16 columns of them: by column, warp and row
};

template <int D, int M>
constexpr size_t smem_bytes() {
  return Layout<D, M>::kCtl + (M == kQ8Few ? sizeof(CtlFew) : M != kBf16 ? sizeof(CtlQ8) : sizeof(Ctl));
}
static_assert(smem_bytes<128, kBf16>() <= 232448 && smem_bytes<128, kQ8>() <= 232448 && smem_bytes<128, kStaged>() <= 232448 &&
              smem_bytes<128, kQ8Few>() <= 232448 && smem_bytes<64, kBf16>() <= 232448, "");

// Waits for the phase of `bar` with this parity, at most kWaitNs from the block's last sign of life in
// exact_row; false once the block gives up.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, Ctl* ctl, int32_t* status) {
  volatile uint32_t *abort = &ctl->abort, *beat = &ctl->beat;
  uint64_t t0 = globaltimer();
  uint32_t b0 = *beat;
  while (!mbar_try(bar, parity)) {
    if (*abort) return false;
    const uint32_t b = *beat;
    if (b != b0) {
      b0 = b;
      t0 = globaltimer();
    }
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

// One arrival for the warp, after all its lanes' work so far.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A ring position: entry and the parity of its current filling.
template <int N>
struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void step() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// K and V tiles pass through a ring in the order in which the MMA warp needs and releases them.  A
// segment's n position tiles are its 2 n entries: with two tiles of rows K0 V0 K1 V1 .., with two streams
// K0 K1 V0 K2 V1 K3 .. V(n-2) V(n-1).  (Loaded as K0 V0 K1 V1 there too, V tiles waited in the ring for two
// position tiles: one row, 64 tiles a block from HBM, 98.7 us instead of 96.6.)
__host__ __device__ __forceinline__ constexpr int entry_of(const Segment& g, int v, int j) {
  if (g.two) return 2 * j + v;
  const int k = 2 * j - 1, w = 2 * j + 2, last = 2 * g.n - 1;
  return v ? (w < last ? w : last) : k > 0 ? k : 0;
}
// and back: whether entry i is a V tile, and of which position tile
__host__ __device__ __forceinline__ constexpr int tile_of(const Segment& g, int i, int& v) {
  if (g.two) {
    v = i & 1;
    return i >> 1;
  }
  v = i == 2 * g.n - 1 || (i > 0 && !(i & 1));
  return !v ? (i + 1) >> 1 : i == 2 * g.n - 1 ? g.n - 1 : (i - 2) >> 1;
}

// A ring of N stages filled by two producers, one of K and one of V tiles.  Each waits for the release of entry
// e - N by its parity, which is sound only if entry e - 2N is known to be released.  It is, as long as entries are
// released in order and a producer's own entry before e is e - N or later: it waited for that one's turn, e - 2N or
// later.  (Released out of order, or with fewer stages, a producer could pass a phase early, fill a stage twice and
// overflow its barrier.)  Whether these two orders keep to that, within segments and from one to the next:
__host__ __device__ constexpr bool ring_holds(int N) {
  for (int kinds = 0; kinds < 4; ++kinds)
    for (int lens = 0; lens < 36; ++lens) {
      int last[2] = {0, 0}, c0 = 0;
      for (int k = 0; k < 2; ++k) {
        Segment g = {};
        g.two = (kinds >> k) & 1;
        g.n = 1 + (k ? lens / 6 : lens % 6);
        for (int i = 0; i < 2 * g.n; ++i) {
          int v = 0;
          const int j = tile_of(g, i, v);
          if (j < 0 || j >= g.n || entry_of(g, v, j) != i) return false;
        }
        for (int v = 0; v < 2; ++v)
          for (int j = 0; j < g.n; ++j) {
            const int e = c0 + entry_of(g, v, j);
            if (k + j > 0 && (e <= last[v] || e - last[v] > N)) return false;
            last[v] = e;
          }
        c0 += 2 * g.n;
      }
    }
  return true;
}

// --------------------------------------------------------------------------- one row, plainly
// Row r, query head h by one warp: 32 positions at a time, a lane per position for the scores,
// D/32 dims per lane for the output; fp32, and no position beyond the row's own is touched.
// `beat`: counted every 1024 positions (the rest of the block may be waiting), or NULL.
template <int D, int M>
__device__ __noinline__ void exact_row(const AttnParams& p, int r, int h, volatile uint32_t* beat) {
  const int lane = threadIdx.x & 31, kvh = h / p.plan.G, s = seq_of_row(p.seqs, r);
  const int n = p.seqs.len[s] - p.seqs.row0[s + 1] + r + 1;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + static_cast<size_t>(r) * p.q_stride + static_cast<size_t>(h) * D);
  const uint16_t* kv16 = reinterpret_cast<const uint16_t*>(p.kv);
  const int8_t* codes = reinterpret_cast<const int8_t*>(p.kv);
  const __half* scales = reinterpret_cast<const __half*>(p.kv + p.code_bytes);
  const float c = 1.4426950408889634f * rsqrtf(static_cast<float>(D));
  float m = -INFINITY, sum = 0.f, o[D / 32];
  uint32_t seen = 0;                                 // positions whose page is in range
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int t0 = 0; t0 < n; t0 += 32) {
    if (beat != nullptr && lane == 0 && t0 % 1024 == 0) *beat = *beat + 1;
    const int t = t0 + lane;
    int64_t line = -1;
    float x = -INFINITY;
    if (t < n) {
      const int page = __ldg(p.bt + static_cast<size_t>(s) * p.maxpg + t / p.ps);
      if (page >= 0 && page < p.P) {
        line = (static_cast<int64_t>(page) * 2 * p.plan.Hkv + kvh) * p.ps + t % p.ps;
        x = 0.f;
#pragma unroll 4
        for (int d = 0; d < D / 8; ++d) {            // 8 dims at a time
          const uint4 a = __ldg(q + d);
          const uint32_t qw[4] = {a.x, a.y, a.z, a.w};
          float k[8];
          if constexpr (M != kBf16) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + line * D) + d);
            const float sc = __half2float(scales[line * (D / 32) + d / 4]);
#pragma unroll
            for (int e = 0; e < 8; ++e) k[e] = static_cast<float>(static_cast<int8_t>((e < 4 ? w.x : w.y) >> (8 * (e % 4)))) * sc;
          } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(kv16 + line * D) + d);
            const uint32_t kw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) k[e] = e & 1 ? bf_hi(kw[e / 2]) : bf_lo(kw[e / 2]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x = fmaf(e & 1 ? bf_hi(qw[e / 2]) : bf_lo(qw[e / 2]), k[e], x);
        }
        x *= c;
      }
    }
    float mx = x;
#pragma unroll
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
    mx = fmaxf(mx, m);
    // (a row whose scores so far are all -inf or NaN takes 0 as its reference; NaN goes on into w)
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float f = m == -INFINITY ? 0.f : ex2(m - ref), w = line >= 0 ? ex2(x - ref) : 0.f;
    float ws = w;
#pragma unroll
    for (int k = 16; k; k >>= 1) ws += __shfl_xor_sync(~0u, ws, k);
    sum = (sum == 0.f ? 0.f : sum * f) + ws;
    m = mx;
    seen |= __ballot_sync(~0u, line >= 0);
    // A NaN in the sum (all lanes') stays, and makes every dim NaN: the rest of the row changes nothing.  (A NaN in
    // an early key is every row's: a 4096-token prompt of 16 heads took 41 ms, now 0.31.)
    if (sum != sum) break;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] == 0.f ? 0.f : o[i] * f;
    for (uint32_t in = __ballot_sync(~0u, line >= 0); in; in &= in - 1) {
      const int j = __ffs(in) - 1;
      const int64_t lv = __shfl_sync(~0u, line, j) + static_cast<int64_t>(p.plan.Hkv) * p.ps;
      const float wj = __shfl_sync(~0u, w, j);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int d = 32 * i + lane;
        float v;
        if constexpr (M != kBf16) v = static_cast<float>(codes[lv * D + d]) * __half2float(scales[lv * (D / 32) + i]);
        else v = bf_lo(kv16[lv * D + d]);
        o[i] = fmaf(wj, v, o[i]);
      }
    }
  }
  // (positions, but every score -inf: 0 / 0, the NaN that the formula has)
  uint16_t* out = p.out + (static_cast<size_t>(r) * p.Hq + h) * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    out[32 * i + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(seen == 0u ? 0.f : o[i] / sum));
}

// --------------------------------------------------------------------------- loads (warp 8: K, warp 11: V)
// A tile of 16-position pages takes 8 copies (q8_0: 16), which a warp issues one by one, so K and V have a
// warp each (64 position tiles a block, one row, the cache in L2: bf16 85 us with one warp, 59 with
// two; q8_0 126 and 100).  They share a ring (see ring_holds), whose entries the MMA warp (raw stages: the
// decode warps) releases in order.
template <int D, int M>
__device__ __forceinline__ void produce(const AttnParams& p, uint32_t base, Ctl* ctl, int only) {
  using L = Layout<D, M>;
  static_assert(M == kQ8Few || ring_holds(M == kQ8 ? L::kRawStages : L::kStages), "");   // (kQ8Few: a raw ring each)
  const int lane = threadIdx.x & 31;
  const int r = p.box, nbox = kTile / r;                       // copies of a tile
  const bool mine = lane < nbox;
  SegmentWalk walk(p.plan, blockIdx.x);
  Segment g;
  uint32_t jg = 0, c0 = 0;                                     // position tiles and ring entries so far
  for (; walk.next(p.plan, p.seqs, g); c0 += 2 * g.n) {
    const int32_t* bt = p.bt + static_cast<size_t>(g.s) * p.maxpg;
    // lane b looks up the page of the tile's b-th copy, one tile ahead
    auto lookup = [&](int j) {
      const int pos = (g.tile0 + j) * kTile + lane * r;
      return j < g.n && mine && pos < g.len ? __ldg(bt + pos / p.ps) : -1;
    };
    int page_next = lookup(0);
    for (int j = 0; j < g.n; ++j, ++jg) {
      const int page = page_next;
      page_next = lookup(j + 1);
      const int pos = (g.tile0 + j) * kTile + lane * r;
      const bool good = mine && page >= 0 && page < p.P;
      if (mine && pos < g.len && !good && p.status) *p.status = MK_ERR_DEVICE_BOUNDS;
      const uint32_t ok = __ballot_sync(~0u, good);
      uint32_t mask = 0;                                       // a bit per 8 positions
      if (only == 0 || M == kQ8Few) mask = __ballot_sync(~0u, lane < 16 && ((ok >> (lane * 8 / r)) & 1u));
      if (only == 0 && lane == 0) ctl->mask[jg % kMasks] = mask;
      const uint32_t e = c0 + entry_of(g, only, j);
      if constexpr (M == kStaged) {
        // whole tiles of the workspace, their positions out of range or behind the sequence zeros already
        const uint32_t st = e % L::kStages, bar = smem_u32(&ctl->full[st]);
        if (!mbar_wait(smem_u32(&ctl->empty[st]), ((e / L::kStages) & 1u) ^ 1u, ctl, p.status)) return;
        if (lane == 0) {
          mbar_expect(bar, L::kTileBytes);
          tma_5d(base + L::kKv + st * L::kTileBytes, &p.map, g.kvh * (kTile / 8),
                 (p.stage0[g.s] + g.tile0 + j) * 2 + only, bar);
        }
        __syncwarp();
      } else if constexpr (M == kBf16) {
        const uint32_t st = e % L::kStages, bar = smem_u32(&ctl->full[st]);
        if (!mbar_wait(smem_u32(&ctl->empty[st]), ((e / L::kStages) & 1u) ^ 1u, ctl, p.status)) return;
        if (lane == 0) mbar_expect(bar, L::kTileBytes);
        __syncwarp();
        // a copy out of the pool's range fills its positions with zeros
        if (mine)
          tma_5d(base + L::kKv + st * L::kTileBytes + lane * (r / 8) * L::kGroup, &p.map,
                 (g.kvh * p.ps + pos % p.ps) / 8, (good ? page : p.P) * 2 + only, bar);
      } else {
        // one ring of raw stages by entries, or K's and V's by position tiles
        const uint32_t ring = M == kQ8Few ? kRawFew : L::kRawStages, at = M == kQ8Few ? jg : e;
        const uint32_t rs = at % ring + (M == kQ8Few ? only * kRawFew : 0);
        const uint32_t bar = smem_u32(&ctl->raw_full[rs]), dst = base + L::kRaw + rs * kRawBytes;
        if (!mbar_wait(smem_u32(&ctl->raw_empty[rs]), ((at / ring) & 1u) ^ 1u, ctl, p.status)) return;
        if (lane == 0) {
          if constexpr (M == kQ8Few) static_cast<CtlFew*>(ctl)->raw_mask[rs] = mask;
          mbar_expect(bar, __popc(ok) * r * 136);
        }
        __syncwarp();
        if (good) {
          const size_t line = (static_cast<size_t>(page) * 2 + only) * p.plan.Hkv * p.ps +
                            static_cast<size_t>(g.kvh) * p.ps + pos % p.ps;
          bulk_g2s(dst + lane * r * 128, p.kv + line * 128, r * 128, bar);
          bulk_g2s(dst + kTile * 128 + lane * r * 8, p.kv + p.code_bytes + line * 8, r * 8, bar);
        }
      }
    }
  }
}

// What a page holds behind the sequence's last position must not meet a weight, not even a zero one
// (0 * NaN): zeros go there in a segment's last V tile.  (q8_0 tiles are zeroed as they are decoded;
// whole copies behind the sequence are zeros already.)
template <int M>
__device__ __forceinline__ bool trims(const Segment& g) { return M == kBf16 && (g.tile0 + g.n) * kTile > g.len; }

// Warp 10.  Query tiles: TT tokens x G heads x 64 dims a box, as soon as the last S of the segment
// before has read the tiles -- under that segment's last softmax, values and epilogue.  And the trim
// of a segment's last V tile, when the MMA warp, which keeps the entry until then, says that it landed.
template <int D, int M>
__device__ __forceinline__ void produce_q(const AttnParams& p, uint32_t base, Ctl* ctl) {
  using L = Layout<D, M>;
  const int lane = threadIdx.x & 31;
  SegmentWalk walk(p.plan, blockIdx.x);
  Segment g;
  uint32_t k = 0, trimmed = 0, c0 = 0;
  while (walk.next(p.plan, p.seqs, g)) {
    if (k > 0 && !mbar_wait(smem_u32(&ctl->qfree), (k - 1) & 1, ctl, p.status)) return;
    ++k;
    if (M == kQ8Few && lane == 0) {                // the rows four times, once for each warp of a warpgroup
      const uint32_t bar = smem_u32(&ctl->qraw[0]), rows = kFew / p.plan.G * p.plan.G;
      mbar_expect(bar, 4 * rows * D * 2);
      for (int w = 0; w < 4; ++w)
        for (int h = 0; h < D / 64; ++h)
          tma_4d(base + h * kTile * 128 + w * kFew * 128, &p.qmap, h, g.kvh * p.plan.G, p.seqs.row0[g.s] + g.tok0, bar);
    } else if (lane == 0) {
      for (int t = 0; t < (g.two ? 2 : 1); ++t) {
        const uint32_t bar = smem_u32(&ctl->qraw[t]);
        mbar_expect(bar, p.plan.TT * p.plan.G * D * 2);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_4d(base + t * L::kTileBytes + h * kTile * 128, &p.qmap, h, g.kvh * p.plan.G,
                 p.seqs.row0[g.s] + g.tok0 + t * p.plan.TT, bar);
      }
    }
    __syncwarp();
    const uint32_t c = c0 + 2 * g.n - 1;
    c0 += 2 * g.n;
    if (trims<M>(g)) {
      if (!mbar_wait(smem_u32(&ctl->landed), trimmed & 1, ctl, p.status)) return;
      ++trimmed;
      const int first = g.len - (g.tile0 + g.n - 1) * kTile, last = (first + p.box - 1) / p.box * p.box;
      const uint32_t v = base + L::kKv + c % L::kStages * L::kTileBytes + (lane / 8 % (D / 64)) * 1024 + (lane & 7) * 16;
      for (int n = first + lane / (D / 8); n < last; n += 256 / D) sts16(v + (n >> 3) * L::kGroup + (n & 7) * 128, 0, 0, 0, 0);
      fence_async_smem();
      warp_arrive(smem_u32(&ctl->trim));
    }
  }
}

// --------------------------------------------------------------------------- q8_0 (warps 12-15)
// Codes to fp16 operand tiles.  With its sign bit flipped a code byte is code + 128, and as the low
// byte of 0x64.. the fp16 1024 + 128 + code; less 1152 that is the code exactly, times the scale
// rounded once.  Positions of pages out of range or behind the sequence become zeros, values of a
// scale of 512 or more NaN: 128 (a code may be -128) times the next smaller one, 511.75, is fp16's largest.
//
// kQ8Few has two groups of four warps: one decodes K tiles (group 0), one V tiles, each from raw stages of
// its own.  They share the operand ring as the two loaders do over a bf16 cache, and by the same argument.
constexpr uint32_t kMaxScale = 0x5fffu;            // 511.75, of which and below the values are decoded
template <int D, int M>
__device__ __forceinline__ void decode(const AttnParams& p, uint32_t base, Ctl* ctl, int group) {
  using L = Layout<D, M>;
  static_assert(M != kQ8Few || ring_holds(L::kStages), "");
  const int tid = threadIdx.x & 127;
  // A thread takes chunks x and x ^ 8 (8 codes, 16 bytes of operand each) of rows tid/8 + 16 i:
  // odd rows begin with the upper half, which keeps 8-byte reads and 16-byte writes free of conflicts.
  const int row0 = tid >> 3, x = (tid & 7) | (row0 & 1) << 3;
  constexpr int NR = kTile / 16;                    // rows of a thread
  // the four scales of a row to the pairs (d, d) of its chunks' blocks of 32: one permute each
  const uint32_t b0 = x >> 2, pick0 = 0x1010u + b0 * 0x2222u, pick1 = 0x1010u + (b0 ^ 2u) * 0x2222u;
  const __half2 bias = __half2half2(__float2half_rn(1152.f));
  // raw stage rs to operand stage st: a tile whose page mask is given and of which `left` positions are the sequence's
  auto work = [&](uint32_t rs, uint32_t st, uint32_t mask, int left) {
    // row0 + 16 i is in group 2 i + row0 / 8 of 8 rows, at row0 % 8 of it
    const uint32_t src = base + L::kRaw + rs * kRawBytes + row0 * 128;
    const uint32_t ssrc = base + L::kRaw + rs * kRawBytes + kTile * 128 + row0 * 8;
    const uint32_t dst = base + L::kKv + st * L::kTileBytes + (row0 >> 3) * L::kGroup + (row0 & 7) * 128 +
                         (((x & 7) ^ (row0 & 7)) << 4);
    // every load before the first store: the stores are what a load would wait behind
    uint32_t w[NR][4], sc[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(src + i * 2048 + x * 8));
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i][2]), "=r"(w[i][3]) : "r"(src + i * 2048 + (x ^ 8) * 8));
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(sc[i][0]), "=r"(sc[i][1]) : "r"(ssrc + i * 128));
    }
    // (kQ8Few: the loader may go on before the codes are worked on)
    if constexpr (M == kQ8Few) warp_arrive(smem_u32(&ctl->raw_empty[rs]));
    // Most tiles need neither zeros nor NaN: every position is the sequence's, and no scale has the top bit of its
    // exponent (is 2 or more).  A warp that sees so leaves the tests out, a third of its instructions (one
    // token at 262144: 81.3 -> 71.9 us).  With units of more rows it is not the decode that they wait for.
    auto convert = [&](auto all) {
      constexpr bool ALL = decltype(all)::value;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const bool live = ALL || (((mask >> (2 * i + (row0 >> 3))) & 1u) && row0 + 16 * i < left);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t d = __byte_perm(sc[i][0], sc[i][1], c == 0 ? pick0 : pick1);
          if constexpr (!ALL) {
            d = (d & 0x7fffu) > kMaxScale ? 0x7fff7fffu : d;
            d = live ? d : 0u;
          }
          const __half2 dd = *reinterpret_cast<const __half2*>(&d);
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t v = w[i][2 * c + k] ^ 0x80808080u;
            uint32_t a = __byte_perm(v, 0x64646464u, 0x4140), b = __byte_perm(v, 0x64646464u, 0x4342);
            const __half2 ha = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&a), bias), dd);
            const __half2 hb = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&b), bias), dd);
            o[2 * k] = *reinterpret_cast<const uint32_t*>(&ha);
            o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&hb);
          }
          sts16(dst + i * 2 * L::kGroup + (((x >> 3) ^ c) << 10), o[0], o[1], o[2], o[3]);
        }
      }
    };
    bool plain = false;
    if constexpr (M == kQ8Few) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NR; ++i) top |= sc[i][0] | sc[i][1];
      plain = mask == 0xffffu && left >= kTile && !__any_sync(~0u, (top & 0x40004000u) != 0u);
    }
    if (plain) convert(std::true_type());
    else convert(std::false_type());
    if constexpr (M == kQ8) warp_arrive(smem_u32(&ctl->raw_empty[rs]));
    fence_async_smem();
    warp_arrive(smem_u32(&ctl->full[st]));
  };
  SegmentWalk walk(p.plan, blockIdx.x);
  Segment g;
  if constexpr (M == kQ8) {
    Ring<L::kStages> ring;
    Ring<L::kRawStages> raw;
    uint32_t jg = 0;
    for (; walk.next(p.plan, p.seqs, g); jg += g.n) {
      for (int i = 0; i < 2 * g.n; ++i) {
        int v;
        const int j = tile_of(g, i, v);
        if (!mbar_wait(smem_u32(&ctl->raw_full[raw.st]), raw.ph, ctl, p.status)) return;
        if (!mbar_wait(smem_u32(&ctl->empty[ring.st]), ring.ph ^ 1u, ctl, p.status)) return;
        work(raw.st, ring.st, ctl->mask[(jg + j) % kMasks], g.len - (g.tile0 + j) * kTile);
        raw.step();
        ring.step();
      }
    }
  } else {
    Ring<kRawFew> raw;
    for (uint32_t c0 = 0; walk.next(p.plan, p.seqs, g); c0 += 2 * g.n) {
      for (int j = 0; j < g.n; ++j) {
        const uint32_t e = c0 + entry_of(g, group, j), st = e % L::kStages, rs = raw.st + group * kRawFew;
        if (!mbar_wait(smem_u32(&ctl->raw_full[rs]), raw.ph, ctl, p.status)) return;
        if (!mbar_wait(smem_u32(&ctl->empty[st]), ((e / L::kStages) & 1u) ^ 1u, ctl, p.status)) return;
        work(rs, st, static_cast<CtlFew*>(ctl)->raw_mask[rs], g.len - (g.tile0 + j) * kTile);
        raw.step();
      }
    }
  }
}

// --------------------------------------------------------------------------- MMAs (warp 9)
// A wait that gives up does not leave the loops (their bounds stay uniform that way): in an aborted block
// every later wait returns at once and the products are of whatever is there.  All of tensor memory is the
// block's, from column 0: S (and P, over it) of tile (stream) t at column t * 128, O at 256 + t * D.
template <int D, int M>
__device__ __forceinline__ void issue(const AttnParams& p, uint32_t base, Ctl* ctl) {
  using L = Layout<D, M>;
  constexpr uint32_t kIdS = tc_idesc(M == kBf16, kTile, kTile, false), kIdO = tc_idesc(M == kBf16, kTile, D, true);
  constexpr uint32_t kHiQ = desc_hi(1024), kHiKv = desc_hi(L::kGroup);
  constexpr uint32_t kStep = L::kTileBytes >> 4;   // a tile in descriptor units
  const uint32_t q_lo = desc_lo(base, 16), k_lo = desc_lo(base + L::kKv, 16), v_lo = desc_lo(base + L::kKv, 1024);
  uint32_t c0 = 0;                                 // ring entry of the segment's first K tile
  uint32_t pp = 0, qq = 0, tr = 0;                 // phases of pfull and of the query tiles (a bit for each t), and trim
  const int lane = threadIdx.x & 31;
  auto wait = [&](const uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    if (!mbar_try(a, parity)) mbar_wait_slow(a, parity, ctl, p.status);
    __syncwarp();
  };
  auto wait_full = [&](uint32_t c) { wait(&ctl->full[c % L::kStages], (c / L::kStages) & 1); };
  auto release = [&](uint32_t c) { tc_commit(smem_u32(&ctl->empty[c % L::kStages])); };
  auto scores = [&](int t, int qt, uint32_t c) {   // S of tile (stream) t from Q tile qt and the K tile in entry c
    const uint32_t a = q_lo + qt * kStep, b = k_lo + c % L::kStages * kStep;
    tc_after();
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      mma_ss(t * kTile, a + (k / 4) * (kTile * 128 >> 4) + (k % 4) * 2, kHiQ, b + (k / 4) * (1024 >> 4) + (k % 4) * 2, kHiKv,
             kIdS, k > 0);
    tc_commit(smem_u32(&ctl->sfull[t]));
    // the page mask travels with an ordinary arrival: the warp that wrote it arrived on `full`
    if (lane == 0) mbar_arrive(smem_u32(&ctl->sfull[t]));
    __syncwarp();
  };
  // O of tile (stream) t += P times the V tile in entry c, each half of P as it comes
  auto values = [&](int t, uint32_t c, bool acc) {
    const uint32_t b = v_lo + c % L::kStages * kStep, ph = (pp >> t) & 1;
    pp ^= 1u << t;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      wait(&ctl->pfull[t][h], ph);
      tc_after();
#pragma unroll
      for (int k = 4 * h; k < 4 * h + 4; ++k)
        mma_ts(2 * kTile + t * D, t * kTile + k * 8, b + k * (2 * L::kGroup >> 4), kHiKv, kIdO, acc || k > 0);
    }
  };
  auto wait_q = [&](int t) {
    wait(M != kBf16 ? &ctl->qbar[t] : &ctl->qraw[t], (qq >> t) & 1);
    qq ^= 1u << t;
  };
  auto done_q = [&]() { tc_commit(smem_u32(&ctl->qfree)); };
  SegmentWalk walk(p.plan, blockIdx.x);
  Segment g;
  while (walk.next(p.plan, p.seqs, g)) {
    const uint32_t c = c0;
    auto wait_v = [&](int j) {
      wait_full(c + entry_of(g, 1, j));
      if (j + 1 == g.n && trims<M>(g)) {
        if (lane == 0) mbar_arrive(smem_u32(&ctl->landed));
        wait(&ctl->trim, tr & 1);
        ++tr;
      }
    };
    wait_q(0);
    if (g.two) {
      wait_q(1);
      wait_full(c);
      scores(0, 0, c);
      scores(1, 1, c);
      release(c);
      if (g.n == 1) done_q();
      for (int j = 0; j < g.n; ++j) {
        const bool more = j + 1 < g.n;
        const uint32_t v = c + 2 * j + 1;
        wait_v(j);
        values(0, v, j > 0);
        if (more) {
          wait_full(v + 1);
          scores(0, 0, v + 1);
        }
        values(1, v, j > 0);
        release(v);
        if (more) {
          scores(1, 1, v + 1);
          release(v + 1);
          if (j + 2 == g.n) done_q();
        }
      }
    } else {
      for (int j = 0; j < 2 && j < g.n; ++j) {
        wait_full(c + j);
        scores(j, 0, c + j);
        release(c + j);
      }
      if (g.n <= 2) done_q();
      for (int j = 0; j < g.n; ++j) {
        const int t = j & 1;
        const uint32_t v = c + entry_of(g, 1, j);
        wait_v(j);
        values(t, v, j > 1);
        release(v);
        if (j + 2 < g.n) {                         // the next entry: K of tile j + 2
          wait_full(v + 1);
          scores(t, 0, v + 1);
          release(v + 1);
          if (j + 3 == g.n) done_q();
        }
      }
    }
    tc_commit(smem_u32(&ctl->ofull));
    c0 += 2 * g.n;
  }
}

// --------------------------------------------------------------------------- softmax (warps 0-7)
// q8_0: a thread's landed query row over 2^e as fp16, in place, e the exponent of its largest
// magnitude; returns 2^e.  (Rows of the tile behind the unit's hold anything.)
template <int D, int B>
__device__ __forceinline__ float convert_q(uint32_t tile, int row) {
  constexpr int CH = D / 8;
  auto at = [&](int ch) { return tile + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4); };
  uint32_t w[B][4];                                // B chunks at a time (all of them, or read twice)
  auto load = [&](int c0) {
#pragma unroll
    for (int c = 0; c < B; ++c)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3])
                   : "r"(at(c0 + c)));
  };
  float mx = 0.f;
#pragma unroll
  for (int c0 = 0; c0 < CH; c0 += B) {
    load(c0);
#pragma unroll
    for (int c = 0; c < B; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) mx = max3(mx, fabsf(bf_lo(w[c][k])), fabsf(bf_hi(w[c][k])));
  }
  int e = static_cast<int>(__float_as_uint(mx) >> 23);
  e = e == 0 || e == 255 ? 127 : e == 254 ? 253 : e;       // (zero rows; infinities end in exact_row)
  const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
  for (int c0 = 0; c0 < CH; c0 += B) {
    if (B < CH) load(c0);
#pragma unroll
    for (int c = 0; c < B; ++c) {
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = f16x2(bf_lo(w[c][k]) * down, bf_hi(w[c][k]) * down);
      sts16(at(c0 + c), o[0], o[1], o[2], o[3]);
    }
  }
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

template <int D, int M>
__device__ __forceinline__ void softmax(const AttnParams& p, uint32_t base, Ctl* ctl) {
  const int t = threadIdx.x >> 7, row = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t ts = t * kTile + lane_base, to = 2 * kTile + lane_base;
  constexpr float kBias = M != kBf16 ? 6.f : 0.f;          // weights carry 2^kBias
  SegmentWalk walk(p.plan, blockIdx.x);
  Segment g, next;
  bool have = walk.next(p.plan, p.seqs, g);
  uint32_t phase = 0, jg = 0, seg = 0;             // tiles of this stream, position tiles, segments so far
  uint32_t qs = 0, qr = 0, joins = 0;              // phases of qbar[0], this warpgroup's qraw, and join
  // both warpgroups: what either wrote before is the other's to read
  auto join = [&]() {
    warp_arrive(smem_u32(&ctl->join));
    return mbar_wait(smem_u32(&ctl->join), joins++ & 1, ctl, p.status);
  };
  float cq = p.c;                                  // the row's constant
  // q8_0: the next segment's rows of this warpgroup's tile
  auto take_q = [&](const Segment& n) {
    if constexpr (M != kBf16) {
      if (!n.two && t == 1) return true;
      if (!mbar_wait(smem_u32(&ctl->qraw[t]), qr & 1, ctl, p.status)) return false;
      ++qr;
      cq = p.c * convert_q<D, D / 8>(base + t * Layout<D, M>::kTileBytes, row);
      if (!n.two) static_cast<CtlQ8*>(ctl)->rowc[row] = cq;
      fence_async_smem();
      warp_arrive(smem_u32(&ctl->qbar[t]));
    }
    return true;
  };
  if (have && !take_q(g)) return;
  while (have) {
    const int trows = p.plan.TT * p.plan.G;
    const int urow0 = g.two ? t * trows : 0;       // first row of the tile within the unit
    const int rows = min(trows, g.ntok * p.plan.G - urow0);
    const bool live = row < rows, any = warp * 32 < rows;
    // rows behind the last see everything, so that they never ask for a mask
    const int pos = live ? g.pos0 + ((urow0 + row) * p.plan.by_G >> 16) : INT32_MAX;
    const int mine = g.two ? g.n : (g.n - t + 1) / 2;
    float c = cq;
    if constexpr (M != kBf16) {
      if (!g.two && t == 1 && mine > 0) {          // stream 1 takes the constants of stream 0's rows
        if (!mbar_wait(smem_u32(&ctl->qbar[0]), qs & 1, ctl, p.status)) return;
        c = static_cast<CtlQ8*>(ctl)->rowc[row];
      }
      ++qs;
    }
    const float grow = 8.0f / c;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < mine; ++i) {
      const int j = g.two ? i : 2 * i + t;
      const int limit = pos - (g.tile0 + j) * kTile;           // last column this row sees
      const bool edge = __any_sync(~0u, limit < kTile - 1);
      if (!mbar_wait(smem_u32(&ctl->sfull[t]), phase & 1, ctl, p.status)) return;
      ++phase;
      if (any) {                                   // (warps without rows leave their lanes as they are)
        tc_after();
        const uint32_t mask = ctl->mask[(jg + j) % kMasks];
        float s[kTile];
#pragma unroll
        for (int k = 0; k < kTile; k += 32) tc_ld32(ts + k, s + k);
        tc_wait_ld();
        if (edge) {
#pragma unroll
          for (int k = 0; k < kTile; ++k)
            if (k > limit) s[k] = -INFINITY;
        }
        if (mask != 0xffffu) {
#pragma unroll
          for (int k = 0; k < kTile; ++k)
            if (!((mask >> (k >> 3)) & 1u)) s[k] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int k = 4; k < kTile - 4; k += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[k + e], s[k + 4 + e]);
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], s[kTile - 4], s[kTile - 3]),
                               fmaxf(s[kTile - 2], s[kTile - 1]));
        // The reference moves only when the maximum outgrows it by 2^8: until then weights up to 2^8
        // are as exact in the operands and in fp32 as weights up to 1, and O needs no rescaling.
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
              tc_ld16(to + t * D + k, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float2 x = mul2(make_float2(o[e], o[e + 1]), ff);
                o[e] = x.x;
                o[e + 1] = x.y;
              }
              tc_st16(to + t * D + k, o);
            }
          }
        }
        const float mb = m == -INFINITY ? 0.f : kBias - m * c;
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
            w[k] = M != kBf16 ? f16x2(y.x, y.y) : bf16x2(y.x, y.y);
          }
          // half of P stands when the third quarter is computed (and its own writing is still to come), the
          // rest at the end: the products of the first half start under the second's exponentials
          if (h == 2) {
            tc_wait_st();
            tc_before();
            warp_arrive(smem_u32(&ctl->pfull[t][0]));
          }
          tc_st16(ts + h * 16, w);
          if (h == 3) {
            tc_wait_st();
            tc_before();
            warp_arrive(smem_u32(&ctl->pfull[t][1]));
          }
        }
        const float2 sm = add2(sum[0], sum[1]);
        l += sm.x + sm.y;
      } else {
        warp_arrive(smem_u32(&ctl->pfull[t][0]));
        warp_arrive(smem_u32(&ctl->pfull[t][1]));
      }
    }
    if (!mbar_wait(smem_u32(&ctl->ofull), seg & 1, ctl, p.status)) return;
    tc_after();
    jg += g.n;
    // the next segment's rows, so that its first scores run under this one's epilogue
    have = walk.next(p.plan, p.seqs, next);
    if (have && !take_q(next)) return;

    // m and l in powers of two; a row without a position has m = -inf and l = 0
    m = m == -INFINITY ? m : m * c;
    float f[2] = {g.two && t == 1 ? 0.f : 1.f, g.two && t == 1 ? 1.f : 0.f};
    if (!g.two) {
      // two streams of the same rows: both warpgroups read both outputs, each half of the columns
      ctl->ml[t][row] = make_float2(m, l);
      if (!join()) return;
      const float2 a = ctl->ml[0][row], b = ctl->ml[1][row];
      m = fmaxf(a.x, b.x);
      f[0] = a.x == -INFINITY ? 0.f : ex2(a.x - m);
      f[1] = b.x == -INFINITY ? 0.f : ex2(b.x - m);
      l = a.y * f[0] + b.y * f[1];
    }
    const int urow = urow0 + row;
    const int tok = urow * p.plan.by_G >> 16;
    const int r = p.seqs.row0[g.s] + g.tok0 + tok, h = g.kvh * p.plan.G + urow - tok * p.plan.G;
    // no weight at all: a row without a position, or one whose scores are all -inf or beyond fp32
    bool odd = l == 0.f;
    if (any) {
      // a partial is [D/4][urows] of 4 columns, then [urows] of (m, l): a warp's rows lie side by side
      float4* part = reinterpret_cast<float4*>(p.part + static_cast<size_t>(max(g.slot, 0)) * p.plan.urows * (D + 4));
      // Stores to the output: the four lanes of a quad trade 16-byte pieces, so that each store
      // covers 64 bytes of 8 rows instead of 16 bytes of 32.  The rows of the quad's lanes:
      const int q4 = threadIdx.x & 3;
      uint32_t row_off[4];                         // in heads, from the sequence's first row; ~0: none
#pragma unroll
      for (int e = 0; e < 4; ++e) row_off[e] = __shfl_sync(~0u, live ? static_cast<uint32_t>(r * p.Hq + h) : ~0u, e, 4);
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const int k0 = g.two ? 0 : t * (D / 2), k1 = g.two ? D : k0 + D / 2;
#pragma unroll 1
      for (int k = k0; k < k1; k += 32) {
        float x[32];
        tc_ld32(to + (g.two ? t * D : 0) + k, x);
        tc_wait_ld();
        if (!g.two) {
          if (g.n > 1) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              float y[16];
              tc_ld16(to + D + k + e, y);
              tc_wait_ld();
#pragma unroll
              for (int z = 0; z < 16; ++z) x[e + z] = x[e + z] * f[0] + y[z] * f[1];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] *= f[0];
          }
        }
        if (g.slot >= 0) {
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              part[static_cast<size_t>((k + e) / 4) * p.plan.urows + urow] = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
        } else {
          uint32_t w[4][4];                        // piece e: columns k + 8 e
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float y0 = x[e] * inv, y1 = x[e + 1] * inv;
            odd |= !(fabsf(y0) <= 3.3e38f) || !(fabsf(y1) <= 3.3e38f);
            w[e / 8][e / 2 % 4] = bf16x2(y0, y1);
          }
          // piece e of lane i <-> piece i of lane e, a bit of the index at a time
#pragma unroll
          for (int bit = 1; bit < 4; bit <<= 1) {
            const bool up = (q4 & bit) != 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (e & bit) continue;
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const uint32_t give = up ? w[e][z] : w[e | bit][z];
                const uint32_t got = __shfl_xor_sync(~0u, give, bit);
                if (up) w[e][z] = got;
                else w[e | bit][z] = got;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (row_off[e] != ~0u)
              *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(row_off[e]) * D + k + 8 * q4) =
                  make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
        }
        __syncwarp();
      }
      if (live && g.slot >= 0 && (g.two || t == 0))
        reinterpret_cast<float2*>(part + static_cast<size_t>(D / 4) * p.plan.urows)[urow] = make_float2(m, l);
    }
    // neither stream's next values may overwrite an output that the other warpgroup still reads
    if (!g.two) {
      tc_before();
      if (!join()) return;
    }
    // rows that are not finite, or without a weight, again from the cache, when both warpgroups' columns are
    // written (where both see one they write the same)
    if (g.slot < 0) {
      for (uint32_t todo = __ballot_sync(~0u, odd && live); todo; todo &= todo - 1) {
        const int who = __ffs(todo) - 1;
        const int rr = __shfl_sync(~0u, r, who), hh = __shfl_sync(~0u, h, who);
        __threadfence_block();
        exact_row<D, M>(p, rr, hh, &ctl->beat);
      }
    }
    ++seg;
    g = next;
  }
}

// Units of at most 32 rows over a q8_0 cache (single and speculative tokens).  A row's softmax is one warp's
// work, and with rows in lanes 0-31 alone it is the same warp's, on the scheduler that the decode warps need
// too: half of a position tile's time.  So the rows stand in all four warps' lanes, and warp w takes
// positions 32 w .. 32 w + 31 of each tile: the others' weights are zeros in its lanes, whose O is the sum over its
// own positions.  The eight parts of a row (two streams, four warps), each with its m and l, are
// joined through shared memory.  (One token at 262144 positions, with the two groups of decode warps that the
// saved registers pay for: 87.0 -> 81.3 us.)
template <int D>
__device__ __forceinline__ void softmax_few(const AttnParams& p, uint32_t base, Ctl* ctl) {
  CtlFew* few = static_cast<CtlFew*>(ctl);
  const int t = threadIdx.x >> 7, row = threadIdx.x & 127, lane = row & 31, warp = __shfl_sync(~0u, row >> 5, 0);
  const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t ts = t * kTile + lane_base, to = 2 * kTile + lane_base;
  constexpr float kBias = 6.f;                     // weights carry 2^kBias
  SegmentWalk walk(p.plan, blockIdx.x);
  Segment g, next;
  bool have = walk.next(p.plan, p.seqs, g);
  uint32_t phase = 0, jg = 0, seg = 0, joins = 0, meets = 0;
  auto join = [&]() {                              // both warpgroups
    warp_arrive(smem_u32(&ctl->join));
    return mbar_wait(smem_u32(&ctl->join), joins++ & 1, ctl, p.status);
  };
  auto meet = [&]() {                              // this one
    warp_arrive(smem_u32(&few->shared[t]));
    return mbar_wait(smem_u32(&few->shared[t]), meets++ & 1, ctl, p.status);
  };
  uint32_t taken = 0;
  float cq = p.c;                                  // the row's constant
  auto take_q = [&]() {
    if (!mbar_wait(smem_u32(&ctl->qraw[0]), taken++ & 1, ctl, p.status)) return false;
    cq = p.c * convert_q<D, 4>(base, row);
    few->rowc[row] = cq;
    fence_async_smem();
    warp_arrive(smem_u32(&ctl->qbar[0]));
    return true;
  };
  if (have && t == 0 && !take_q()) return;
  while (have) {
    const int rows = g.ntok * p.plan.G, tok = lane * p.plan.by_G >> 16;
    const bool live = lane < rows;
    // rows behind the last see everything, so that they never ask for a mask
    const int pos = live ? g.pos0 + tok : INT32_MAX;
    const int mine = (g.n - t + 1) / 2;
    float c = cq;
    if (t == 1 && mine > 0) {                      // stream 1 takes the constants of stream 0's rows
      if (!mbar_wait(smem_u32(&ctl->qbar[0]), seg & 1, ctl, p.status)) return;
      c = few->rowc[row];
    }
    const float grow = 8.0f / c;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < mine; ++i) {
      const int j = 2 * i + t;
      const int limit = pos - (g.tile0 + j) * kTile - 32 * warp;   // last of its 32 columns this row sees
      const bool edge = __any_sync(~0u, limit < 31);
      if (!mbar_wait(smem_u32(&ctl->sfull[t]), phase & 1, ctl, p.status)) return;
      ++phase;
      tc_after();
      const uint32_t mask = ctl->mask[(jg + j) % kMasks] >> (4 * warp) & 15u;
      float s[32];
      tc_ld32(ts + 32 * warp, s);
      tc_wait_ld();
      if (edge) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (k > limit) s[k] = -INFINITY;
      }
      if (mask != 15u) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (!((mask >> (k >> 3)) & 1u)) s[k] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int k = 4; k < 28; k += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[k + e], s[k + 4 + e]);
      }
      const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], s[28], s[29]), fmaxf(s[30], s[31]));
      if (i == 0) {
        m = top;
      } else {
        const bool up = top > m + grow;            // (as in softmax)
        if (__any_sync(~0u, up)) {
          const float mn = up ? top : m;
          const float f = m == -INFINITY ? 0.f : ex2((m - mn) * c);
          l *= f;
          m = mn;
          const float2 ff = make_float2(f, f);
#pragma unroll 1
          for (int k = 0; k < D; k += 16) {
            float o[16];
            tc_ld16(to + t * D + k, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 x = mul2(make_float2(o[e], o[e + 1]), ff);
              o[e] = x.x;
              o[e + 1] = x.y;
            }
            tc_st16(to + t * D + k, o);
          }
        }
      }
      const float mb = m == -INFINITY ? 0.f : kBias - m * c;
      const float2 cc = make_float2(c, c), mm = make_float2(mb, mb);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t w[16], none[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 x = fma2(make_float2(s[2 * k], s[2 * k + 1]), cc, mm);
        const float2 y = make_float2(ex2(x.x), ex2(x.y));
        sum[k & 1] = add2(sum[k & 1], y);
        w[k] = f16x2(y.x, y.y);
        none[k] = 0u;
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (h == warp) tc_st16(ts + h * 16, w);
        else tc_st16(ts + h * 16, none);
      }
      tc_wait_st();
      tc_before();
      warp_arrive(smem_u32(&ctl->pfull[t][0]));
      warp_arrive(smem_u32(&ctl->pfull[t][1]));
      const float2 sm = add2(sum[0], sum[1]);
      l += sm.x + sm.y;
    }
    if (!mbar_wait(smem_u32(&ctl->ofull), seg & 1, ctl, p.status)) return;
    tc_after();
    jg += g.n;
    have = walk.next(p.plan, p.seqs, next);
    if (have && t == 0 && !take_q()) return;

    // m and l in powers of two; a part without a position has m = -inf and l = 0
    ctl->ml[t][row] = make_float2(m == -INFINITY ? m : m * c, l);
    if (!join()) return;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, ctl->ml[e >> 2][(e & 3) * 32 + lane].x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 a = ctl->ml[e >> 2][(e & 3) * 32 + lane];
      l += a.x == -INFINITY ? 0.f : a.y * ex2(a.x - m);
    }
    const float m0 = ctl->ml[0][row].x, m1 = ctl->ml[1][row].x;
    const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - m), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
    const int r = p.seqs.row0[g.s] + g.tok0 + tok, h = g.kvh * p.plan.G + lane - tok * p.plan.G;
    float4* part = reinterpret_cast<float4*>(p.part + static_cast<size_t>(max(g.slot, 0)) * p.plan.urows * (D + 4));
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    bool odd = live && g.slot < 0 && l == 0.f;     // (as in softmax)
    // each warpgroup half of the columns, 16 at a time, of which each warp sums up 4
#pragma unroll 1
    for (int k = t * (D / 2); k < (t + 1) * (D / 2); k += 16) {
      float x[16], y[16];
      tc_ld16(to + k, x);
      if (g.n > 1) tc_ld16(to + D + k, y);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) few->part[t][e][warp][lane] = g.n > 1 ? x[e] * f0 + y[e] * f1 : x[e] * f0;
      if (!meet()) return;
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float(*a)[kFew] = few->part[t][4 * warp + e];
        o[e] = a[0][lane] + a[1][lane] + (a[2][lane] + a[3][lane]);
      }
      if (!meet()) return;
      const int col = k + 4 * warp;
      if (live && g.slot >= 0) {
        part[static_cast<size_t>(col / 4) * p.plan.urows + lane] = make_float4(o[0], o[1], o[2], o[3]);
      } else if (live) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] *= inv;
          odd |= !(fabsf(o[e]) <= 3.3e38f);
        }
        *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(r) * p.Hq + h) * D + col) =
            make_uint2(bf16x2(o[0], o[1]), bf16x2(o[2], o[3]));
      }
    }
    if (live && g.slot >= 0 && t == 0 && warp == 0)
      reinterpret_cast<float2*>(part + static_cast<size_t>(D / 4) * p.plan.urows)[lane] = make_float2(m, l);
    // neither stream's next values may overwrite an output that the other warpgroup still reads
    tc_before();
    __threadfence_block();
    if (!join()) return;
    // rows that are not finite, or without a weight, again from the cache (where several warps see one they write
    // the same)
    for (uint32_t todo = __ballot_sync(~0u, odd); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1;
      exact_row<D, kQ8Few>(p, __shfl_sync(~0u, r, who), __shfl_sync(~0u, h, who), &ctl->beat);
    }
    ++seg;
    g = next;
  }
}

template <int D, int M>
__global__ void __launch_bounds__(Layout<D, M>::kThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<D, M>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + L::kCtl);
  const int warp = threadIdx.x >> 5;
  if (base & 1023u) {                              // the operand layouts need it; dynamic shared memory starts so
    if (p.status) *p.status = MK_ERR_UNSUPPORTED;
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {                   // (q8_0: a K or V tile is the decode warps' work)
      mbar_init(smem_u32(&ctl->full[i]), kDecodes<M> ? 4 : 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
      mbar_init(smem_u32(&ctl->raw_full[i]), 1);
      mbar_init(smem_u32(&ctl->raw_empty[i]), 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ctl->qraw[t]), 1);
      mbar_init(smem_u32(&ctl->qbar[t]), 4);
      mbar_init(smem_u32(&ctl->sfull[t]), 2);
      mbar_init(smem_u32(&ctl->pfull[t][0]), 4);
      mbar_init(smem_u32(&ctl->pfull[t][1]), 4);
    }
    mbar_init(smem_u32(&ctl->qfree), 1);
    mbar_init(smem_u32(&ctl->landed), 1);
    mbar_init(smem_u32(&ctl->trim), 1);
    mbar_init(smem_u32(&ctl->ofull), 1);
    mbar_init(smem_u32(&ctl->join), 8);
    if constexpr (M == kQ8Few)
      for (int t = 0; t < 2; ++t) mbar_init(smem_u32(&static_cast<CtlFew*>(ctl)->shared[t]), 4);
    ctl->abort = 0u;
    ctl->beat = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  // (all 512 columns: they begin at column 0, and the roles count on it)
  const uint32_t tm = ctl->tmem;
  if (tm != 0u) {
    if (p.status) *p.status = MK_ERR_UNSUPPORTED;
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
    return;
  }
  // registers follow the work: a softmax thread holds a row of S (the warpgroups' sum is the launch's)
  if (warp < 8) {
    if constexpr (M == kQ8Few) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
      softmax_few<D>(p, base, ctl);
    } else {
      if constexpr (M == kQ8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
      else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      softmax<D, M>(p, base, ctl);
    }
  } else if (warp < 12) {
    if constexpr (kDecodes<M>) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8 || warp == 11) produce<D, M>(p, base, ctl, warp == 8 ? 0 : 1);
    if (warp == 9) issue<D, M>(p, base, ctl);
    if (warp == 10) produce_q<D, M>(p, base, ctl);
  } else if constexpr (kDecodes<M>) {
    if constexpr (M == kQ8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    decode<D, M>(p, base, ctl, (warp - 12) >> 2);
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

// Merges the items that the ranges cut, in block order; blockIdx.x is the item, 2 D threads a block.
// Wide (units of few rows, cut into many parts): a block takes 128 / D rows, a warp every eighth
// partial, whose loads are all on their way before the factors are known.  Else a block takes 8
// rows, a thread 4 columns of one, a warp's 8 rows side by side in a partial; the parts are few.
template <int D, int M, bool WIDE>
__global__ void __launch_bounds__(2 * D) merge_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kWarps = 2 * D / 32, kLanes = D / 4, kRows = WIDE ? 32 / kLanes : 8;
  constexpr int kMine = WIDE ? (kMaxBlocks + kWarps - 1) / kWarps : 1, kAtOnce = 8;
  const AttnPlan& pl = p.plan;
  const int b = pl.cut_block[blockIdx.x], n = pl.cut_parts[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Segment g;
  item_of(pl, p.seqs, pl.start[b + 1].item, g);
  const int rows = g.ntok * pl.G, row0 = blockIdx.y * kRows;
  if (row0 >= rows) return;
  const int lrow = WIDE ? lane / kLanes : lane & 7, chunk = WIDE ? lane % kLanes : warp * 4 + (lane >> 3);
  const int urow = row0 + lrow;
  const bool live = urow < rows;
  const size_t slot = static_cast<size_t>(pl.urows) * (D + 4);
  const float* first = p.part + static_cast<size_t>(2 * b + 1) * slot;            // then slots 2(b+1), 2(b+2), ..
  auto at = [&](int k) { return k == 0 ? first : first + (2 * k - 1) * slot; };
  const size_t at_ml = static_cast<size_t>(pl.urows) * D, at_o = (static_cast<size_t>(chunk) * pl.urows + (live ? urow : 0)) * 4;
  __shared__ float fac[kRows][kMaxBlocks], den[kRows];
  __shared__ float4 sums[WIDE ? kWarps : 1][WIDE ? 32 : 1];
  float4 held[kAtOnce];
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int k = warp + i * kWarps;
      held[i] = k < n ? *reinterpret_cast<const float4*>(at(k) + at_o) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // the factors of each row's partials: a warp a row (D = 64: WIDE's two rows, or two rows a warp in turn)
  for (int r = warp; r < kRows; r += kWarps) {
    const int row = min(row0 + r, rows - 1);
    float top = -INFINITY, L = 0.f;
    for (int k = lane; k < n; k += 32) {
      const float m = at(k)[at_ml + 2 * row];
      fac[r][k] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    for (int k = lane; k < n; k += 32) {
      const float m = fac[r][k], f = m == -INFINITY ? 0.f : ex2(m - top);
      fac[r][k] = f;
      L += f * at(k)[at_ml + 2 * row + 1];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) L += __shfl_xor_sync(~0u, L, o);
    if (lane == 0) den[r] = L;
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4 o, float f) {
    acc.x = fmaf(o.x, f, acc.x);
    acc.y = fmaf(o.y, f, acc.y);
    acc.z = fmaf(o.z, f, acc.z);
    acc.w = fmaf(o.w, f, acc.w);
  };
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (warp + i * kWarps < n) add(held[i], fac[lrow][warp + i * kWarps]);
    for (int i = kAtOnce; i < kMine; ++i) {
      const int k = warp + i * kWarps;
      if (k < n) add(*reinterpret_cast<const float4*>(at(k) + at_o), fac[lrow][k]);
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < kWarps; ++w) add(sums[w][lane], 1.f);
  } else {
#pragma unroll 4
    for (int k = 0; k < n; ++k) add(*reinterpret_cast<const float4*>(at(k) + at_o), fac[lrow][k]);
  }
  const float L = den[lrow], inv = L == 0.f ? 0.f : 1.0f / L;
  const int tok = urow * pl.by_G >> 16;
  const int r = p.seqs.row0[g.s] + g.tok0 + tok, h = g.kvh * pl.G + urow - tok * pl.G;
  acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (live)
    *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(r) * p.Hq + h) * D + chunk * 4) =
        make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
  const float big = fmaxf(fmaxf(fabsf(acc.x), fabsf(acc.y)), fmaxf(fabsf(acc.z), fabsf(acc.w)));
  const bool odd = live && (L == 0.f || !(big <= 3.3e38f) || acc.x != acc.x || acc.y != acc.y || acc.z != acc.z || acc.w != acc.w);
  if constexpr (!WIDE) __syncthreads();            // (a row's columns are several warps')
  uint32_t done = 0;
  for (uint32_t todo = __ballot_sync(~0u, odd); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1;
    const int rr = __shfl_sync(~0u, r, who), hh = __shfl_sync(~0u, h, who), lr = __shfl_sync(~0u, lrow, who);
    if (!((done >> lr) & 1u)) exact_row<D, M>(p, rr, hh, nullptr);
    done |= 1u << lr;
  }
}

// --------------------------------------------------------------------------- staging
// A q8_0 sequence with many units (of query rows) has its cache decoded once, into fp16 tiles in the
// workspace, instead of by every unit's block: tile t of the staged ones is [K, V][KV head][128][D]
// as a page of 128 positions would be.  What Decoder does to a value is done here: the product with
// the scale rounded to fp16, NaN for scales above kMaxScale, zeros for positions out of range or behind the
// sequence.  A thread takes 16 codes: 16 bytes and a scale in, 32 bytes out; HBM bound.
constexpr int kStageThreads = 256;
template <int D>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(const __grid_constant__ AttnParams p, __half* __restrict__ out,
                                                              const __grid_constant__ StageTiles st) {
  constexpr int CH = D / 16, kRows = kStageThreads / CH;       // chunks of a row, rows of a pass
  const int tile = blockIdx.x, vh = blockIdx.y;                // vh: K heads, then V heads
  int i = 0;
  while (i + 1 < st.n && st.first[i + 1] <= tile) ++i;
  const int s = st.seq[i], t = tile - st.first[i], len = p.seqs.len[s];
  const int ch = threadIdx.x % CH;
  const int32_t* bt = p.bt + static_cast<size_t>(s) * p.maxpg;
  uint4 w[kTile / kRows];
  uint16_t sc[kTile / kRows];
#pragma unroll
  for (int k = 0; k < kTile / kRows; ++k) {
    const int pos = t * kTile + k * kRows + threadIdx.x / CH;
    w[k] = make_uint4(0u, 0u, 0u, 0u);
    sc[k] = 0;
    if (pos >= len) continue;
    const int page = __ldg(bt + pos / p.ps);
    if (page < 0 || page >= p.P) {
      if (p.status) *p.status = MK_ERR_DEVICE_BOUNDS;
      continue;
    }
    const size_t line = static_cast<size_t>(page) * 2 * p.plan.Hkv * p.ps + static_cast<size_t>(vh) * p.ps + pos % p.ps;
    w[k] = __ldg(reinterpret_cast<const uint4*>(p.kv + line * D) + ch);
    sc[k] = __ldg(reinterpret_cast<const uint16_t*>(p.kv + p.code_bytes) + line * (D / 32) + ch / 2);
  }
  const __half2 bias = __half2half2(__float2half_rn(1152.f));
#pragma unroll
  for (int k = 0; k < kTile / kRows; ++k) {
    uint32_t d = sc[k];
    if ((d & 0x7fffu) > kMaxScale) d = 0x7fffu;
    const __half2 dd = __half2half2(__ushort_as_half(static_cast<uint16_t>(d)));
    const uint32_t q[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = q[e] ^ 0x80808080u;
      uint32_t lo = __byte_perm(v, 0x64646464u, 0x4140), hi = __byte_perm(v, 0x64646464u, 0x4342);
      const __half2 hl = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&lo), bias), dd);
      const __half2 hh = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&hi), bias), dd);
      o[2 * e] = *reinterpret_cast<const uint32_t*>(&hl);
      o[2 * e + 1] = *reinterpret_cast<const uint32_t*>(&hh);
    }
    uint4* dst = reinterpret_cast<uint4*>(
        out + ((static_cast<size_t>(tile) * 2 * p.plan.Hkv + vh) * kTile + k * kRows + threadIdx.x / CH) * D + 16 * ch);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// --------------------------------------------------------------------------- host
// Sequences whose cache is staged: from kStageUnits units on decoding once is less work than every unit's block
// doing it (a tile staged costs its bytes, 0.017 us of the card a KV head; a unit's block that decodes
// takes 0.8 us longer a tile, 0.005 us of the card); kStageBytes at most are staged in a call.
constexpr int kStageUnits = 6;
constexpr size_t kStageBytes = size_t(1) << 30;

struct CallPlan {
  AttnPlan direct, staged;           // the two launches' (q8_0 only: staged.items may be 0, as direct.items)
  StageTiles tiles;
  int32_t stage0[kMaxSeqs];
  size_t stage_bytes, floats;        // workspace: staged tiles, then partials (the launches follow each other)
  size_t bytes() const { return stage_bytes + floats * sizeof(float); }
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
  return true;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)
                                                                : nullptr;
  }();
  return encode;
}

// bf16 pages (or fp16 tiles of the workspace) to TMA, innermost first: {64 dims, 8 positions, D/64 spans of dims, groups of 8
// positions over the KV heads, pages x (K, V)}.  A box lands as [group][span][8 positions][128 B]:
// 8-position groups a constant distance apart whatever the page size, which is what the operand
// descriptors of both K (rows along dims) and V (rows along positions) need.
int encode_pages(int D_, int heads, int page_size, int pages, bool bf16, const void* kv, int box_pos, CUtensorMap* out) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
  if (!encode) return chunk_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t D = D_, ps = page_size, hkv = heads;
  const cuuint64_t dims[5] = {64, 8, D / 64, hkv * ps / 8, static_cast<cuuint64_t>(pages) * 2};
  const cuuint64_t strides[4] = {D * 2, 128, 8 * D * 2, hkv * ps * D * 2};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(box_pos / 8), 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(kv), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MK_OK : chunk_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
}

// Query rows to TMA: {64 dims, D/64 spans, heads, rows}; a box of TT rows x G heads lands as a tile's
// [row][128 B], rows behind the call's as zeros.
int encode_queries(const mk_cache_shape& c, int G, int tokens, const void* q, int64_t stride, int rows, CUtensorMap* out) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
  if (!encode) return chunk_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t D = c.head_dim;
  const cuuint64_t dims[4] = {64, D / 64, static_cast<cuuint64_t>(c.num_q_heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[3] = {128, D * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MK_OK : chunk_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled (queries) failed (%d)", static_cast<int>(r));
}

// Whether n bytes at `out` share one with `rows` rows of n / rows bytes, `stride` apart, at `q`.  (A row that is
// worked out again reads its query row when its first result is written already.)
bool meets_rows(const void* out, const void* q, uint64_t rows, uint64_t stride, uint64_t n) {
  const uint64_t o = reinterpret_cast<uintptr_t>(out), a = reinterpret_cast<uintptr_t>(q), width = n / rows;
  const uint64_t r = o < a + width ? 0 : (o - a - width) / stride + 1;   // the first row that ends behind o
  return r < rows && a + r * stride < o + n;
}

template <int D, int M>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
  // once per device (a bit each; beyond 64 devices on every call): the attribute is the device's
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(attn_kernel<D, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes<D, M>()));
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  attn_kernel<D, M><<<p.plan.blocks, Layout<D, M>::kThreads, smem_bytes<D, M>(), st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.plan.cuts == 0) return e;
  constexpr int kMerge = M == kBf16 ? kBf16 : kQ8;
  // (plans with units of two tiles cut an item in few parts)
  if (p.plan.urows <= kTile / 2) {
    constexpr int kRows = 128 / D;
    merge_kernel<D, kMerge, true><<<dim3(p.plan.cuts, (p.plan.urows + kRows - 1) / kRows), 2 * D, 0, st>>>(p);
  } else {
    merge_kernel<D, kMerge, false><<<dim3(p.plan.cuts, (p.plan.urows + 7) / 8), 2 * D, 0, st>>>(p);
  }
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
  CallPlan plan;
  if (!plan_call(*shape, seqs, &plan)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  *bytes_out = plan.bytes();
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
  if (q_stride >= int64_t(1) << 38) return chunk_fail(MK_ERR_UNSUPPORTED, "q_stride above 2^38");
  const int rows = p.seqs.row0[num_seqs];
  if (rows > 0 && (!block_tables || !q || !kv_layer || !out))
    return chunk_fail(MK_ERR_INVALID_ARG, "a pointer argument is NULL");
  if (misaligned(block_tables, 4) || misaligned(q, 16) || misaligned(kv_layer, 16) || misaligned(out, 16) ||
      misaligned(workspace, 16))
    return chunk_fail(MK_ERR_INVALID_ARG, "pointers must be 16-byte aligned (block_tables 4-byte)");
  if (rows > 0 && meets_rows(out, q, rows, static_cast<uint64_t>(q_stride) * 2,
                             static_cast<uint64_t>(rows) * c.num_q_heads * c.head_dim * 2))
    return chunk_fail(MK_ERR_INVALID_ARG, "out overlaps q");
  CallPlan plan;
  if (!plan_call(c, p.seqs, &plan)) return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  if (workspace_bytes < plan.bytes() || (plan.bytes() > 0 && !workspace))
    return chunk_fail(MK_ERR_INVALID_ARG, "the workspace holds %zu bytes; these lengths need %zu", workspace_bytes,
                      plan.bytes());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  const bool q8 = (c.flags & MK_FLAG_KV_Q8) != 0;
  p.box = std::min(c.page_size & -c.page_size, kTile);
  p.kv = static_cast<const uint8_t*>(kv_layer);
  p.bt = block_tables;
  p.status = status_out;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.stage_bytes);
  p.code_bytes = static_cast<size_t>(c.num_pages) * 2 * c.num_kv_heads * c.page_size * c.head_dim;
  std::copy(plan.stage0, plan.stage0 + kMaxSeqs, p.stage0);
  p.Hq = c.num_q_heads;
  p.ps = c.page_size;
  p.P = c.num_pages;
  p.maxpg = c.max_pages_per_seq;
  p.c = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(c.head_dim)));
  cudaError_t e = cudaSuccess;
  if (plan.direct.items > 0) {
    p.plan = plan.direct;
    const bool few = q8 && p.plan.urows <= kFew;
    rc = encode_queries(c, p.plan.G, few ? kFew / p.plan.G : p.plan.TT, q, q_stride, rows, &p.qmap);
    if (rc) return rc;
    if (!q8) {
      rc = encode_pages(c.head_dim, c.num_kv_heads, c.page_size, c.num_pages, true, kv_layer, p.box, &p.map);
      if (rc) return rc;
    }
    e = few                 ? launch<128, kQ8Few>(p, st)
        : q8                ? launch<128, kQ8>(p, st)
        : c.head_dim == 128 ? launch<128, kBf16>(p, st)
                            : launch<64, kBf16>(p, st);
  }
  if (e == cudaSuccess && plan.staged.items > 0) {
    p.plan = plan.staged;
    rc = encode_queries(c, p.plan.G, p.plan.TT, q, q_stride, rows, &p.qmap);
    if (!rc) rc = encode_pages(128, c.num_kv_heads, kTile, plan.tiles.first[plan.tiles.n], false, workspace, kTile, &p.map);
    if (rc) return rc;
    stage_kernel<128><<<dim3(plan.tiles.first[plan.tiles.n], 2 * c.num_kv_heads), kStageThreads, 0, st>>>(
        p, static_cast<__half*>(workspace), plan.tiles);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch<128, kStaged>(p, st);
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
