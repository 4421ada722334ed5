// mk_chunk.cu -- a chunk of new tokens into the paged KV cache (mk_append_chunk), cached
// positions back out of it (mk_read_cache), and the argument checks of the chunk operators.
//
// Both kernels move bytes: a row is read once and written once, 16 bytes per thread and access, and
// everything between is in registers.  HBM bounds the bf16 append of 128-wide heads and the read; the q8_0 append
// and heads of 64 are bound by their instructions (see append_kernel).

#include "mk_chunk.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace mk {

void set_last_error(int code, const char* text);

int chunk_fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(code, buf);
  return code;
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int check_chunk(const mk_cache_shape* c, int32_t num_seqs, const int32_t* chunk_lens, const int32_t* seq_lens,
                ChunkSeqs* out) {
  set_last_error(MK_OK, "");
  if (!c) return chunk_fail(MK_ERR_INVALID_ARG, "shape is NULL");
  const struct { const char* n; int32_t v; } pos[] = {
      {"num_q_heads", c->num_q_heads}, {"num_kv_heads", c->num_kv_heads}, {"head_dim", c->head_dim},
      {"page_size", c->page_size}, {"num_pages", c->num_pages}, {"max_pages_per_seq", c->max_pages_per_seq}};
  for (const auto& f : pos)
    if (f.v <= 0) return chunk_fail(MK_ERR_INVALID_ARG, "shape.%s must be > 0 (got %d)", f.n, f.v);
  if (c->flags & ~MK_FLAG_KV_Q8) return chunk_fail(MK_ERR_INVALID_ARG, "unknown bits in shape.flags");
  if (c->num_q_heads % c->num_kv_heads)
    return chunk_fail(MK_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  if (c->head_dim != 64 && c->head_dim != 128) return chunk_fail(MK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->num_q_heads / c->num_kv_heads > 8)
    return chunk_fail(MK_ERR_UNSUPPORTED, "more than 8 query heads per KV head");
  if (c->page_size % 8) return chunk_fail(MK_ERR_UNSUPPORTED, "page_size must be a multiple of 8");
  if ((c->flags & MK_FLAG_KV_Q8) && c->head_dim != 128)
    return chunk_fail(MK_ERR_UNSUPPORTED, "the q8_0 KV cache needs head_dim 128");
  const int64_t max_len = static_cast<int64_t>(c->max_pages_per_seq) * c->page_size;
  if (max_len > (int64_t(1) << 30)) return chunk_fail(MK_ERR_UNSUPPORTED, "max_pages_per_seq*page_size above 2^30");
  if (c->num_q_heads > 1024) return chunk_fail(MK_ERR_UNSUPPORTED, "more than 1024 query heads");
  const int64_t page_rows = static_cast<int64_t>(c->num_kv_heads) * 2 * c->page_size;   // below 2^42
  if (page_rows > INT32_MAX / c->num_pages)
    return chunk_fail(MK_ERR_UNSUPPORTED, "the layer's KV pool has 2^31 or more rows");
  if (num_seqs < 1 || num_seqs > kMaxSeqs) return chunk_fail(MK_ERR_INVALID_ARG, "num_seqs outside 1..%d", kMaxSeqs);
  if (!chunk_lens || !seq_lens) return chunk_fail(MK_ERR_INVALID_ARG, "chunk_lens or seq_lens is NULL");
  int64_t rows = 0;
  out->n = num_seqs;
  for (int s = 0; s < num_seqs; ++s) {
    if (chunk_lens[s] < 0 || seq_lens[s] < chunk_lens[s] || seq_lens[s] > max_len)
      return chunk_fail(MK_ERR_INVALID_ARG,
                        "sequence %d: not 0 <= chunk_len (%d) <= seq_len (%d) <= max_pages_per_seq*page_size", s,
                        chunk_lens[s], seq_lens[s]);
    out->row0[s] = static_cast<int32_t>(rows);
    out->len[s] = seq_lens[s];
    rows += chunk_lens[s];
    if (rows * c->num_q_heads >= (int64_t(1) << 31) || rows >= (int64_t(1) << 24))
      return chunk_fail(MK_ERR_UNSUPPORTED, "too many rows in one call");
  }
  out->row0[num_seqs] = static_cast<int32_t>(rows);
  return MK_OK;
}

int clear_status(int32_t* status_out, cudaStream_t s) {
  if (!status_out) return MK_OK;
  if (misaligned(status_out, 4)) return chunk_fail(MK_ERR_INVALID_ARG, "status_out must be 4-byte aligned");
  const cudaError_t e = cudaMemsetAsync(status_out, 0, sizeof(int32_t), s);
  return e == cudaSuccess ? MK_OK : chunk_fail(MK_ERR_CUDA, "status word: %s", cudaGetErrorString(e));
}

namespace {

constexpr int kBlock = 128;
constexpr int kMaxTile = 64;
constexpr int kMaxPairs = 64;   // rotated pairs of a head

struct Cache {
  uint8_t* kv;
  const int32_t* bt;
  int32_t* status;
  int32_t Hkv, ps, P, maxpg;
  size_t code_bytes;            // q8_0: the code plane
};

// Frequencies as 64-bit fixed-point fractions of a turn per position.  position * turns wraps
// modulo one turn exactly, so the angle of a far position is reduced without a rounding: what is
// left is the frequency's own error (2^-53 of it) times the position, as in a 64-bit angle.
struct Turns {
  uint64_t f[kMaxPairs];
};

__device__ __forceinline__ void unpack8(const uint4 w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
// the larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// The cache row (within the layer's [P][2][Hkv][ps] rows of K) of packed row r, -1 for a page out
// of range.
__device__ __forceinline__ int32_t slot_of_row(const ChunkSeqs& q, const Cache& c, int r, int* pos_out) {
  const int s = seq_of_row(q, r);
  const int pos = q.len[s] - q.row0[s + 1] + r;
  *pos_out = pos;
  const int32_t page = __ldg(c.bt + static_cast<size_t>(s) * c.maxpg + pos / c.ps);
  if (page < 0 || page >= c.P) {
    if (c.status) *c.status = MK_ERR_DEVICE_BOUNDS;
    return -1;
  }
  return page * 2 * c.Hkv * c.ps + pos % c.ps;
}

// Dims [8*ca, 8*ca+8) and [8*cb, ..) of a head belong to lane l of its D/16 lanes.  Half layout:
// pairs (i, i + R/2) meet in one lane (chunks l and l + R/16); behind the rotated dims, and in
// the interleaved layout throughout, chunks 2l and 2l+1.
__device__ __forceinline__ void lane_chunks(int l, int R, bool half, int& ca, int& cb) {
  const bool h = half && l < R / 16;
  ca = h ? l : 2 * l;
  cb = h ? l + R / 16 : 2 * l + 1;
}

// A warp takes a row, or a quarter or half of its heads where rows are few: it computes the row's
// cos and sin (two pairs a lane) and passes them around once, so that each lane holds those of its 8
// pairs for all the heads.  D/16 lanes take a head: two 16-byte loads, the norm's sum by shuffles, the
// rotation in registers, two 16-byte stores (q8_0: 8-byte codes and, per head, one 8-byte store of its
// four scales); the loads of the next kFly heads are in flight meanwhile.  Reads 2 B and writes 2 B
// (17/16 B) a value.  Over bf16 with heads of 128 that bounds it; over q8_0 it is the instructions, of which the
// shuffles of norms and maxima wait longest (4112 tokens with norms, one wave of blocks: 20 us in the profiler, DRAM
// at 27 %), and with heads of 64 too (16384 tokens of 18 heads: 18.5 us, 27 %).  (With the angles read from shared memory for every head, waiting for
// those reads was the most frequent stall: 33.1 us for 8192 tokens of 32 + 2 * 4 heads, now 28.4, 5.9 TB/s.)
template <int D, bool Q8>
__global__ void __launch_bounds__(kBlock) append_kernel(const __grid_constant__ ChunkSeqs seqs,
                                                        const __grid_constant__ Cache c,
                                                        const __grid_constant__ Turns turns, int T, int Hq,
                                                        const uint16_t* __restrict__ qkv, int64_t stride, int R,
                                                        int interleaved, float mscale, const uint16_t* q_norm,
                                                        const uint16_t* k_norm, float eps,
                                                        uint16_t* __restrict__ q_out) {
  constexpr int LH = D / 16, kWarps = kBlock / 32;   // lanes of a head
  // loads in flight against registers (and with them warps): 8192 bf16 tokens of 40 heads of 128 took 31.7,
  // 29.9, 28.4 us at 1, 2, 3; 16384 of 18 heads of 64 took 16.8, 16.4, 17.3; 4112 q8_0 tokens 17.6, 19.8, 20.0
  constexpr int kFly = Q8 ? 1 : D == 128 ? 3 : 2;
  __shared__ float2 cs[kWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LH;
  const int share = kWarps / T;                    // warps of a row
  const int r = blockIdx.x * T + warp / share;
  if (r >= seqs.row0[seqs.n]) return;
  const int H = Hq + 2 * c.Hkv, step = share * (32 / LH);
  const uint16_t* const src = qkv + static_cast<size_t>(r) * stride;
  int h = (warp % share) * (32 / LH) + lane / LH;
  uint4 wa[kFly], wb[kFly];
  auto fetch = [&](int i, int h) {
    if (h >= H) return;
    int ca, cb;
    lane_chunks(l, R, !interleaved && h < Hq + c.Hkv, ca, cb);
    wa[i] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(h) * D + 8 * ca));
    wb[i] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(h) * D + 8 * cb));
  };
#pragma unroll
  for (int i = 0; i < kFly; ++i) fetch(i, h + i * step);
  int pos;
  const int32_t slot = slot_of_row(seqs, c, r, &pos);
  float2 tr[8];                                    // of the lane's pairs, in the order it meets them
  if (R > 0) {
    for (int p = lane; p < R / 2; p += 32) {
      const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * turns.f[p]);    // [-1/2, 1/2) of a turn
      float sn, co;
      sincospif(static_cast<float>(turn) * 1.0842021724855044e-19f, &sn, &co);               // turn * 2^-63 half turns
      cs[warp][p] = make_float2(co * mscale, sn * mscale);
    }
    __syncwarp();
    if (l < R / 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) tr[i] = cs[warp][8 * l + i];   // both layouts: pairs 8 l .. 8 l + 7
    }
  }
  for (; h < H; h += kFly * step) {
#pragma unroll
   for (int fly = 0; fly < kFly; ++fly) {
    const int ch = h + fly * step;
    if (ch >= H) break;                            // (the lanes of a head agree; the shuffles below are theirs)
    const bool isq = ch < Hq, isv = ch >= Hq + c.Hkv;
    int ca, cb;
    lane_chunks(l, R, !interleaved && !isv, ca, cb);
    float a[8], b[8];
    unpack8(wa[fly], a);
    unpack8(wb[fly], b);
    fetch(fly, ch + kFly * step);
    const uint16_t* gain = isq ? q_norm : k_norm;
    if (!isv) {
      // the lanes of a head are in one warp and agree on it (a warp's last heads may be missing:
      // whole heads, so the mask is theirs)
      if (gain != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
        const uint32_t m = ((1u << LH) - 1u) << (lane / LH * LH);
#pragma unroll
        for (int o = 1; o < LH; o <<= 1) ss += __shfl_xor_sync(m, ss, o);
        const float rs = rsqrtf(ss / D + eps);
        float ga[8], gb[8];
        unpack8(*reinterpret_cast<const uint4*>(gain + 8 * ca), ga);
        unpack8(*reinterpret_cast<const uint4*>(gain + 8 * cb), gb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = a[i] * rs * ga[i];
          b[i] = b[i] * rs * gb[i];
        }
      }
      if (l < R / 16) {
        if (interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = tr[i], y = tr[4 + i];
            const float a0 = a[2 * i], b0 = b[2 * i];
            a[2 * i] = a0 * x.x - a[2 * i + 1] * x.y;
            a[2 * i + 1] = a[2 * i + 1] * x.x + a0 * x.y;
            b[2 * i] = b0 * y.x - b[2 * i + 1] * y.y;
            b[2 * i + 1] = b[2 * i + 1] * y.x + b0 * y.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = tr[i];
            const float a0 = a[i];
            a[i] = a0 * x.x - b[i] * x.y;
            b[i] = b[i] * x.x + a0 * x.y;
          }
        }
      }
    }
    if (isq) {
      uint16_t* dst = q_out + (static_cast<size_t>(r) * Hq + ch) * D;
      *reinterpret_cast<uint4*>(dst + 8 * ca) = pack8(a);
      *reinterpret_cast<uint4*>(dst + 8 * cb) = pack8(b);
      continue;
    }
    if (slot < 0) continue;                        // the whole row's
    const int kvh = isv ? ch - Hq - c.Hkv : ch - Hq;
    const size_t line = static_cast<size_t>(slot) + static_cast<size_t>(isv ? c.Hkv + kvh : kvh) * c.ps;
    if constexpr (!Q8) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(c.kv) + line * D;
      *reinterpret_cast<uint4*>(dst + 8 * ca) = pack8(a);
      *reinterpret_cast<uint4*>(dst + 8 * cb) = pack8(b);
    } else {
      // the largest magnitude of each 32-value block over the head's lanes; a NaN is the largest, and so the
      // block's scale: all of it is then NaN, whatever the codes (under an infinite scale none is finite)
      float m[4] = {0.f, 0.f, 0.f, 0.f};
      float ma = 0.f, mb = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ma = max_nan(ma, fabsf(a[i]));
        mb = max_nan(mb, fabsf(b[i]));
      }
      const uint32_t mask = ((1u << LH) - 1u) << (lane / LH * LH);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = max_nan(ca / 4 == k ? ma : 0.f, cb / 4 == k ? mb : 0.f);
#pragma unroll
        for (int o = 1; o < LH; o <<= 1) m[k] = max_nan(m[k], __shfl_xor_sync(mask, m[k], o));
      }
      // the step's quantizer: d = max/127 in fp32, codes by its fp32 reciprocal (ties away from
      // zero), d stored as f16
      uint8_t* codes = c.kv + line * D;
      uint16_t* scales = reinterpret_cast<uint16_t*>(c.kv + c.code_bytes) + line * (D / 32);
      float d4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) d4[k] = m[k] / 127.0f;
      auto put = [&](const float (&x)[8], int ch) {
        const int k = ch / 4;
        const float d = k == 0 ? d4[0] : k == 1 ? d4[1] : k == 2 ? d4[2] : d4[3];
        const float id = d != 0.f ? 1.0f / d : 0.f;
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint8_t q = static_cast<uint8_t>(static_cast<int8_t>(roundf(x[i] * id)));
          w[i / 4] |= static_cast<uint32_t>(q) << (8 * (i % 4));
        }
        *reinterpret_cast<uint2*>(codes + 8 * ch) = make_uint2(w[0], w[1]);
      };
      put(a, ca);
      put(b, cb);
      if (l == 0) {
        const __half2 lo = __floats2half2_rn(d4[0], d4[1]), hi = __floats2half2_rn(d4[2], d4[3]);
        *reinterpret_cast<uint2*>(scales) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
  }
}

// One block takes T rows; a thread takes 16 bytes of one head's K or V row (8 bf16 values, or 16
// codes with their block's scale) and neighbouring threads the row's next, kUnroll of them at a
// time so that their loads are in flight together.  Bytes in, bytes out: HBM bound.
constexpr int kUnroll = 4, kReadUnits = 4;   // at a time; a thread's in all (16: 67 us where 4 take 59, 131072 q8_0 positions)
template <int D, bool Q8>
__global__ void __launch_bounds__(kBlock) read_kernel(const __grid_constant__ ChunkSeqs seqs,
                                                      const __grid_constant__ Cache c, int T,
                                                      uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out) {
  __shared__ int32_t slot[kMaxTile];
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * T, nr = min(T, seqs.row0[seqs.n] - r0);
  if (tid < nr) {
    int pos;
    slot[tid] = slot_of_row(seqs, c, r0 + tid, &pos);
  }
  __syncthreads();
  constexpr int VAL = Q8 ? 16 : 8, CH = D / VAL;
  const int heads = 2 * c.Hkv, ch = tid % CH;   // units: [row][K heads, V heads][chunk]
  constexpr int kStep = kBlock / CH;            // heads between a thread's units
  int row = 0, hh = tid / CH;
  auto wrap = [&]() {
    while (hh >= heads) {
      hh -= heads;
      ++row;
    }
  };
  wrap();
  while (row < nr) {
    uint4 w[kUnroll];
    uint16_t sc[kUnroll];
    int urow[kUnroll], uh[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      urow[i] = row;
      uh[i] = hh;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      sc[i] = 0;
      if (row < nr && slot[row] >= 0) {
        const size_t line = static_cast<size_t>(slot[row]) + static_cast<size_t>(hh) * c.ps;
        w[i] = __ldg(reinterpret_cast<const uint4*>(c.kv + line * D * (Q8 ? 1 : 2)) + ch);
        if constexpr (Q8) sc[i] = __ldg(reinterpret_cast<const uint16_t*>(c.kv + c.code_bytes) + line * (D / 32) + ch / 2);
      }
      hh += kStep;
      wrap();
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (urow[i] >= nr) break;
      const bool isv = uh[i] >= c.Hkv;
      uint16_t* dst = (isv ? v_out : k_out) +
                      (static_cast<size_t>(r0 + urow[i]) * c.Hkv + (isv ? uh[i] - c.Hkv : uh[i])) * D + VAL * ch;
      if constexpr (!Q8) {
        *reinterpret_cast<uint4*>(dst) = w[i];
      } else {
        const float d = __half2float(__ushort_as_half(sc[i]));
        const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            f[k] = static_cast<float>(static_cast<int8_t>(q[2 * half + k / 4] >> (8 * (k % 4)))) * d;
          reinterpret_cast<uint4*>(dst)[half] = pack8(f);
        }
      }
    }
  }
}

Cache cache_of(const mk_cache_shape& s, const int32_t* bt, const void* kv, int32_t* status) {
  Cache c;
  c.kv = static_cast<uint8_t*>(const_cast<void*>(kv));
  c.bt = bt;
  c.status = status;
  c.Hkv = s.num_kv_heads;
  c.ps = s.page_size;
  c.P = s.num_pages;
  c.maxpg = s.max_pages_per_seq;
  c.code_bytes = static_cast<size_t>(s.num_pages) * 2 * s.num_kv_heads * s.page_size * s.head_dim;
  return c;
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MK_OK : chunk_fail(MK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_rope_frequencies(int32_t rotary_dim, double theta, double factor, int32_t original_len,
                                   double beta_fast, double beta_slow, double* inv_freq_out) {
  set_last_error(MK_OK, "");
  if (rotary_dim < 2 || rotary_dim % 2) return chunk_fail(MK_ERR_INVALID_ARG, "rotary_dim must be a positive even number");
  if (!(theta > 1.0) || !std::isfinite(theta)) return chunk_fail(MK_ERR_INVALID_ARG, "theta must be above 1 and finite");
  if (!(factor >= 1.0) || !std::isfinite(factor)) return chunk_fail(MK_ERR_INVALID_ARG, "factor must be at least 1 and finite");
  if (original_len < 0) return chunk_fail(MK_ERR_INVALID_ARG, "original_len is negative");
  if (original_len > 0 && !(beta_fast > beta_slow && beta_slow > 0.0 && std::isfinite(beta_fast)))
    return chunk_fail(MK_ERR_INVALID_ARG, "not beta_fast > beta_slow > 0");
  if (!inv_freq_out) return chunk_fail(MK_ERR_INVALID_ARG, "inv_freq_out is NULL");
  const double two_pi = 6.283185307179586476925;
  double lo = 0.0, hi = 0.0;
  if (original_len > 0) {
    // the (real) pair index that turns beta times within original_len positions:
    // original_len * theta^(-2i/R) / (2 pi) = beta
    auto index = [&](double beta) {
      return rotary_dim * std::log(original_len / (beta * two_pi)) / (2.0 * std::log(theta));
    };
    lo = std::fmax(std::floor(index(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(index(beta_slow)), rotary_dim - 1.0);
    if (!(hi > lo)) hi = lo + 0.001;   // a step instead of a ramp
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / rotary_dim);
    double keep = 0.0;   // share of the unscaled frequency
    if (original_len > 0) keep = 1.0 - std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
    inv_freq_out[i] = f * keep + f / factor * (1.0 - keep);
  }
  return MK_OK;
}

extern "C" int mk_append_chunk(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                               const int32_t* seq_lens, const int32_t* block_tables, const void* qkv,
                               int64_t qkv_stride, const mk_rope* rope, const void* q_norm, const void* k_norm,
                               float eps, void* q_out, void* kv_layer, int32_t* status_out, mk_stream_t stream) {
  ChunkSeqs seqs;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (rc) return rc;
  const mk_cache_shape& c = *shape;
  const int D = c.head_dim, H = c.num_q_heads + 2 * c.num_kv_heads;
  int R = 0, inter = 0;
  float mscale = 1.f;
  Turns turns = {};
  if (rope && rope->rotary_dim != 0) {
    R = rope->rotary_dim;
    inter = rope->interleaved;
    mscale = rope->mscale;
    if (R < 0 || R % 16 || R > D)
      return chunk_fail(MK_ERR_INVALID_ARG, "rotary_dim must be 0 or a multiple of 16 up to head_dim (got %d)", R);
    if (inter != 0 && inter != 1) return chunk_fail(MK_ERR_INVALID_ARG, "rope.interleaved must be 0 or 1");
    if (!std::isfinite(mscale)) return chunk_fail(MK_ERR_INVALID_ARG, "rope.mscale is not finite");
    if (!rope->inv_freq) return chunk_fail(MK_ERR_INVALID_ARG, "rope.inv_freq is NULL");
    for (int i = 0; i < R / 2; ++i) {
      const double f = rope->inv_freq[i];
      if (!std::isfinite(f)) return chunk_fail(MK_ERR_INVALID_ARG, "rope.inv_freq[%d] is not finite", i);
      double t = f / 6.283185307179586476925;
      t -= std::floor(t);                                       // [0, 1], 1 only by rounding
      turns.f[i] = t < 1.0 ? static_cast<uint64_t>(std::ldexp(t, 64)) : 0u;
    }
  }
  if (!(eps >= 0.f) || !std::isfinite(eps)) return chunk_fail(MK_ERR_INVALID_ARG, "eps must be >= 0 and finite");
  if (qkv_stride < static_cast<int64_t>(H) * D || qkv_stride % 8)
    return chunk_fail(MK_ERR_INVALID_ARG, "qkv_stride must be a multiple of 8, at least (Hq + 2*Hkv)*head_dim");
  const int rows = seqs.row0[num_seqs];
  if (rows > 0 && (!block_tables || !qkv || !q_out || !kv_layer))
    return chunk_fail(MK_ERR_INVALID_ARG, "a pointer argument is NULL");
  if (misaligned(block_tables, 4) || misaligned(qkv, 16) || misaligned(q_out, 16) || misaligned(kv_layer, 16) ||
      misaligned(q_norm, 16) || misaligned(k_norm, 16))
    return chunk_fail(MK_ERR_INVALID_ARG, "pointers must be 16-byte aligned (block_tables 4-byte)");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  const Cache cache = cache_of(c, block_tables, kv_layer, status_out);
  const int T = rows >= 4 * 304 ? 4 : rows >= 2 * 304 ? 2 : 1;   // two blocks an SM before a warp takes more heads
  const int grid = (rows + T - 1) / T;
  auto go = [&](auto kernel) {
    kernel<<<grid, kBlock, 0, st>>>(seqs, cache, turns, T, c.num_q_heads, static_cast<const uint16_t*>(qkv), qkv_stride,
                                    R, inter, mscale, static_cast<const uint16_t*>(q_norm),
                                    static_cast<const uint16_t*>(k_norm), eps, static_cast<uint16_t*>(q_out));
  };
  if (c.flags & MK_FLAG_KV_Q8) go(append_kernel<128, true>);
  else if (D == 128) go(append_kernel<128, false>);
  else go(append_kernel<64, false>);
  return launched("append");
}

extern "C" int mk_read_cache(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                             const int32_t* seq_lens, const int32_t* block_tables, const void* kv_layer, void* k_out,
                             void* v_out, int32_t* status_out, mk_stream_t stream) {
  ChunkSeqs seqs;
  int rc = check_chunk(shape, num_seqs, chunk_lens, seq_lens, &seqs);
  if (rc) return rc;
  const mk_cache_shape& c = *shape;
  const int rows = seqs.row0[num_seqs];
  if (rows > 0 && (!block_tables || !kv_layer || !k_out || !v_out))
    return chunk_fail(MK_ERR_INVALID_ARG, "a pointer argument is NULL");
  if (misaligned(block_tables, 4) || misaligned(kv_layer, 16) || misaligned(k_out, 16) || misaligned(v_out, 16))
    return chunk_fail(MK_ERR_INVALID_ARG, "pointers must be 16-byte aligned (block_tables 4-byte)");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  const Cache cache = cache_of(c, block_tables, kv_layer, status_out);
  const int per = 2 * c.num_kv_heads * c.head_dim / ((c.flags & MK_FLAG_KV_Q8) ? 16 : 8);   // units of a row
  int T = kReadUnits * kBlock / per;
  T = T < 1 ? 1 : T > kMaxTile ? kMaxTile : T;
  while (T > 1 && (rows + T - 1) / T < 304) T = (T + 1) / 2;                                 // two blocks an SM first
  const int grid = (rows + T - 1) / T;
  auto go = [&](auto kernel) {
    kernel<<<grid, kBlock, 0, st>>>(seqs, cache, T, static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out));
  };
  if (c.flags & MK_FLAG_KV_Q8) go(read_kernel<128, true>);
  else if (c.head_dim == 128) go(read_kernel<128, false>);
  else go(read_kernel<64, false>);
  return launched("read");
}
