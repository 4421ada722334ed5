// mk_chunk_attn.cu -- causal attention of a chunk of new tokens over the paged KV cache
// (mk_chunk_attention).

#include "mk_chunk.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

namespace mk {
namespace {

constexpr int kWarps = 4;

struct AttnParams {
  ChunkSeqs seqs;
  const uint8_t* kv;
  const int32_t* bt;
  int32_t* status;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  size_t code_bytes;
  int32_t Hq, Hkv, ps, P, maxpg;
  float scale;
};

__device__ __forceinline__ float bf(uint16_t u) { return __uint_as_float(static_cast<uint32_t>(u) << 16); }

// One warp per (row, query head): 32 positions at a time, a lane per position for the scores and
// D/32 dims per lane for the output; one pass with the running maximum and sum of the softmax.
template <int D, bool Q8>
__global__ void __launch_bounds__(32 * kWarps) attn_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float qs[kWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int rows = p.seqs.row0[p.seqs.n];
  if (unit >= static_cast<int64_t>(rows) * p.Hq) return;
  const int r = static_cast<int>(unit / p.Hq), h = static_cast<int>(unit % p.Hq), kvh = h / (p.Hq / p.Hkv);
  const int s = seq_of_row(p.seqs, r);
  const int n = p.seqs.len[s] - p.seqs.row0[s + 1] + r + 1;   // positions this row sees
  for (int d = lane; d < D; d += 32) qs[warp][d] = bf(p.q[r * p.q_stride + h * D + d]) * p.scale;
  __syncwarp();
  float m = -INFINITY, sum = 0.f, o[D / 32] = {};
  for (int t0 = 0; t0 < n; t0 += 32) {
    const int t = t0 + lane;
    int64_t line = -1;
    float x = -INFINITY;
    if (t < n) {
      const int page = p.bt[static_cast<size_t>(s) * p.maxpg + t / p.ps];
      if (page >= 0 && page < p.P) {
        line = (static_cast<int64_t>(page) * 2 * p.Hkv + kvh) * p.ps + t % p.ps;
        x = 0.f;
        for (int d = 0; d < D; ++d) {
          float k;
          if constexpr (Q8)
            k = static_cast<float>(reinterpret_cast<const int8_t*>(p.kv)[line * D + d]) *
                __half2float(reinterpret_cast<const __half*>(p.kv + p.code_bytes)[line * (D / 32) + d / 32]);
          else
            k = bf(reinterpret_cast<const uint16_t*>(p.kv)[line * D + d]);
          x = fmaf(qs[warp][d], k, x);
        }
      } else if (p.status) {
        *p.status = MK_ERR_DEVICE_BOUNDS;
      }
    }
    float mx = x;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
    mx = fmaxf(mx, m);
    if (mx == -INFINITY) continue;   // no position yet
    const float c = __expf(m - mx), w = line >= 0 ? __expf(x - mx) : 0.f;
    float ws = w;
    for (int k = 16; k; k >>= 1) ws += __shfl_xor_sync(~0u, ws, k);
    sum = sum * c + ws;
    m = mx;
    for (int i = 0; i < D / 32; ++i) o[i] *= c;
    for (int j = 0; j < 32; ++j) {
      const int64_t lj = __shfl_sync(~0u, line, j);
      const float wj = __shfl_sync(~0u, w, j);
      if (lj < 0) continue;
      const int64_t lv = lj + static_cast<int64_t>(p.Hkv) * p.ps;
      for (int i = 0; i < D / 32; ++i) {
        const int d = 32 * i + lane;
        float v;
        if constexpr (Q8)
          v = static_cast<float>(reinterpret_cast<const int8_t*>(p.kv)[lv * D + d]) *
              __half2float(reinterpret_cast<const __half*>(p.kv + p.code_bytes)[lv * (D / 32) + i]);
        else
          v = bf(reinterpret_cast<const uint16_t*>(p.kv)[lv * D + d]);
        o[i] = fmaf(wj, v, o[i]);
      }
    }
  }
  for (int i = 0; i < D / 32; ++i) {
    const float v = sum > 0.f ? o[i] / sum : sum == 0.f ? 0.f : o[i] + sum;   // NaN stays NaN
    p.out[(static_cast<size_t>(r) * p.Hq + h) * D + 32 * i + lane] =
        __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
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
  *bytes_out = 0;
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = clear_status(status_out, st);
  if (rc || rows == 0) return rc;
  p.kv = static_cast<const uint8_t*>(kv_layer);
  p.bt = block_tables;
  p.status = status_out;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<uint16_t*>(out);
  p.code_bytes = static_cast<size_t>(c.num_pages) * 2 * c.num_kv_heads * c.page_size * c.head_dim;
  p.Hq = c.num_q_heads;
  p.Hkv = c.num_kv_heads;
  p.ps = c.page_size;
  p.P = c.num_pages;
  p.maxpg = c.max_pages_per_seq;
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.head_dim)));
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(rows) * p.Hq + kWarps - 1) / kWarps);
  if (c.flags & MK_FLAG_KV_Q8) attn_kernel<128, true><<<grid, 32 * kWarps, 0, st>>>(p);
  else if (c.head_dim == 128) attn_kernel<128, false><<<grid, 32 * kWarps, 0, st>>>(p);
  else attn_kernel<64, false><<<grid, 32 * kWarps, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MK_OK : chunk_fail(MK_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
}
