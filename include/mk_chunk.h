/*
 * mk_chunk.h -- operators on chunks of new tokens over the paged KV cache (device work).
 *
 * mk_decode_step decodes one token per row.  These calls are the cache's other side: they
 * take a CHUNK of new tokens per sequence -- a whole prompt, a slice of one, speculative
 * tokens, one token, or a ragged mix of all of these -- over the pages and block tables of
 * one layer, the same ones the step, mk_kv_pool and mk_paged_attention_noalloc use:
 *   mk_append_chunk     per-head RMSNorm of q and k, rotary positions, the cache write
 *   mk_chunk_attention  causal attention of the new tokens over their sequences' positions
 *   mk_read_cache       cached positions back as contiguous bf16 rows
 * A layer's prefill is: QKV product, mk_append_chunk, mk_chunk_attention, the rest of the
 * layer; the decode steps then go on from the same cache.
 *
 * Common arguments
 *   shape         host struct, the layer's heads and pages
 *   num_seqs      sequences of the call, 1..64
 *   chunk_lens    HOST int32 [num_seqs]: rows (new tokens) of each sequence, >= 0
 *   seq_lens      HOST int32 [num_seqs]: its length INCLUDING them (>= chunk_lens[s], at most
 *                 max_pages_per_seq*page_size); row i of sequence s is at position
 *                 seq_lens[s] - chunk_lens[s] + i
 *   block_tables  device int32 [num_seqs][max_pages_per_seq]; entries past
 *                 ceil(seq_len/page_size) are not read
 *   kv_layer      device, the pages of ONE layer: bf16 [num_pages][2 (K,V)][num_kv_heads]
 *                 [page_size][head_dim], or one layer of the q8_0 layout (MK_FLAG_KV_Q8)
 *   status_out    device int32 [1] or NULL; receives MK_OK, or MK_ERR_DEVICE_BOUNDS if a block
 *                 table entry that the call needs was outside 0..num_pages-1.  Such pages are
 *                 never touched (see each call).  With NULL the report is lost.
 * Rows are packed: sequence s owns rows chunk_lens[0]+..+chunk_lens[s-1] and on.  Rows of
 * outputs behind the last sequence's are left as they were.
 *
 * Conventions are mk.h's: arguments are checked before anything is launched, work is enqueued
 * on `stream` of the current device and the call returns at once; host arrays are read during
 * the call; nothing is allocated and nothing synchronises, so calls can be captured into CUDA
 * graphs (a replay uses the lengths of the capture).  There is no shared state: calls on
 * different streams may overlap as long as their outputs and workspaces do not.  Pointers must
 * be 16-byte aligned (block_tables and status_out: 4-byte).
 *
 * Limits (MK_ERR_UNSUPPORTED beyond): head_dim 64 or 128, at most 1024 query heads and 8 per KV head,
 * page_size a multiple of 8, max_pages_per_seq*page_size <= 2^30, num_pages*2*num_kv_heads*
 * page_size < 2^31, fewer than 2^24 rows; the q8_0 cache needs head_dim 128.
 */
#ifndef MK_CHUNK_H
#define MK_CHUNK_H

#include <stddef.h>
#include <stdint.h>

#include "mk.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mk_cache_shape {
  int32_t num_q_heads;
  int32_t num_kv_heads; /* divides num_q_heads; query head h reads KV head h / (num_q_heads/num_kv_heads) */
  int32_t head_dim;
  int32_t page_size;         /* tokens per page */
  int32_t num_pages;         /* pages of the pool */
  int32_t max_pages_per_seq; /* row length of the block table */
  int32_t flags;             /* 0 or MK_FLAG_KV_Q8 */
} mk_cache_shape;

/* Rotary positions: pair i of a head is turned by position * inv_freq[i] and scaled by mscale. */
typedef struct mk_rope {
  int32_t rotary_dim;     /* first dims of the head that are rotated: 0, or a multiple of 16 up to head_dim */
  int32_t interleaved;    /* 0: pair i is dims (i, i + rotary_dim/2); 1: dims (2i, 2i+1) */
  const double* inv_freq; /* HOST [rotary_dim/2] radians per position; the engine's step uses theta^(-2i/D) */
  float mscale;           /* factor of the rotated dims (1 for none) */
} mk_rope;

/*
 * Frequencies for mk_rope: inv_freq_out[i] = theta^(-2i/rotary_dim), HOST [rotary_dim/2], and
 * for contexts `factor` times longer than the model's original_len positions (factor > 1):
 *   original_len == 0: every frequency divided by factor (positions interpolated);
 *   original_len > 0:  by parts -- a pair that turns at least beta_fast times within
 *                      original_len positions is kept, one that turns at most beta_slow times
 *                      is divided by factor, and between the two the frequency goes linearly
 *                      from one to the other with the number of turns' place in the pair index
 *                      (the index at which a pair turns beta times is real-valued; the ramp runs
 *                      between floor and ceil of the two, kept inside 0..rotary_dim-1).
 * Errors: MK_ERR_INVALID_ARG (rotary_dim not a positive even number, theta <= 1 or not finite,
 * factor < 1, original_len < 0, with original_len > 0 not beta_fast > beta_slow > 0, NULL output).
 */
int mk_rope_frequencies(int32_t rotary_dim, double theta, double factor, int32_t original_len, double beta_fast,
                        double beta_slow, double* inv_freq_out);

/*
 * Take the new tokens' fused QKV rows into the cache.
 *   qkv:         device bf16 [rows][qkv_stride]; a row holds num_q_heads, then num_kv_heads k, then
 *                num_kv_heads v heads of head_dim values; qkv_stride in elements, a multiple of 8
 *   rope:        host struct or NULL (no rotation)
 *   q_norm, k_norm: device bf16 [head_dim] or NULL: x * rsqrt(mean(x^2) + eps) * gain over each head
 *                of q / of k, before the rotation
 *   q_out:       device bf16 [rows][num_q_heads][head_dim], the query rows mk_chunk_attention takes
 * k (normed and rotated) and v are written to their positions of kv_layer: as bf16, or quantized
 * from their fp32 values as MK_FLAG_KV_Q8 describes.  What is not finite stays so: a bf16 value as
 * it is, a q8_0 block of 32 with a NaN or an infinity among its values gets a NaN or infinite scale, so
 * that none of it reads back as finite (the step's own quantizer passes over a NaN).  Everything
 * is computed in fp32 (the angle of far positions exactly reduced) and rounded once.  A row whose
 * page is out of range writes q_out but no k or v.  Two rows must not write one position (pages
 * shared by two sequences may be read, not appended to).  qkv, q_out and kv_layer must not overlap.
 */
int mk_append_chunk(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens, const int32_t* seq_lens,
                    const int32_t* block_tables, const void* qkv, int64_t qkv_stride, const mk_rope* rope,
                    const void* q_norm, const void* k_norm, float eps, void* q_out, void* kv_layer,
                    int32_t* status_out, mk_stream_t stream);

/*
 * Bytes of device workspace that mk_chunk_attention needs for these lengths (0 when it needs
 * none), written to bytes_out.  Host only.  It holds the partial outputs of contexts split over
 * blocks (at most 42 MB) and, for q8_0 sequences with many new tokens, their cache decoded to fp16
 * (4 bytes a position, KV head and dim; at most 1 GiB in a call).
 */
int mk_chunk_attention_workspace(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                                 const int32_t* seq_lens, size_t* bytes_out);

/*
 * out[r][h] = softmax attention (scale 1/sqrt(head_dim)) of q[r][h] over positions 0..p of its
 * sequence, p the row's own position; the new tokens' k and v must be in the cache already.
 *   q:         device bf16 [rows][q_stride]: num_q_heads heads of head_dim; q_stride in elements, a
 *              multiple of 8 (num_q_heads*head_dim when contiguous)
 *   out:       device bf16 [rows][num_q_heads][head_dim]; overlaps no row of q (MK_ERR_INVALID_ARG), nor kv_layer
 *   workspace: device, at least mk_chunk_attention_workspace bytes (NULL if 0), contents lost; a
 *              call owns it until its work is done
 * Products run on the tensor cores: over a bf16 cache with bf16 operands (the softmax weights are
 * rounded to bf16), over a q8_0 cache with fp16 ones (weights, decoded values and scaled query rows
 * are rounded to fp16; rows that fp16 cannot hold are computed in fp32 instead).  Scores, softmax
 * statistics and outputs are accumulated in fp32 and rounded once.
 * Rows never see later positions, whatever NaN or infinity these hold.  Scores beyond fp32's range
 * count as infinite: +inf makes its row NaN, -inf is no weight, and a row whose scores are all -inf is
 * NaN.  Every row that NaN or infinity reaches, or fp16 cannot hold, costs an fp32 pass over its
 * positions (up to its first NaN score): an 8192-token prompt may take a thousand times as long.
 * Pages out of range are skipped: a row attends over its other positions, and one that has none gets
 * zeros.  What lies in a page behind a sequence's last position is never used, whatever its bits.
 * A device wait that runs out (a fault of the library) leaves outputs unfinished and is reported as
 * MK_ERR_TIMEOUT in status_out.
 */
int mk_chunk_attention(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens,
                       const int32_t* seq_lens, const int32_t* block_tables, const void* q, int64_t q_stride,
                       const void* kv_layer, void* out, void* workspace, size_t workspace_bytes, int32_t* status_out,
                       mk_stream_t stream);

/*
 * The last chunk_lens[s] positions of each sequence as contiguous rows: k_out and v_out, device
 * bf16 [rows][num_kv_heads][head_dim] (a q8_0 value is code * scale, rounded once).  With
 * chunk_lens == seq_lens that is every position.  Rows of pages out of range are zeros.  The outputs
 * overlap neither each other nor kv_layer.
 */
int mk_read_cache(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens, const int32_t* seq_lens,
                  const int32_t* block_tables, const void* kv_layer, void* k_out, void* v_out, int32_t* status_out,
                  mk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MK_CHUNK_H */
