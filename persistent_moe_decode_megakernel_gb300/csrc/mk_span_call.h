// mk_span_call.h -- mk_window_attention and mk_prefix_attention for callers that allocate: as mk_chunk.h declares them, with
// a function that is asked for the workspace where a call needs one.  Asking for its size first (..._workspace) and then
// calling makes the call's plan twice, 4 to 16 us each on an x86 host.
#ifndef MK_SPAN_CALL_H
#define MK_SPAN_CALL_H

#include "../../include/mk_chunk.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mk_span_workspace {
  void* ptr; /* given: device memory of `bytes` bytes, or NULL */
  size_t bytes;
  void* (*take)(void* ctx, size_t bytes); /* or NULL; asked at most once, for > 0 bytes; NULL from it: MK_ERR_OOM.  Throws nothing */
  void* ctx;
} mk_span_workspace;

int mk_window_attention_in(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens, const int32_t* seq_lens,
                           int32_t window, int32_t sinks, const int32_t* block_tables, const void* q, int64_t q_stride,
                           const void* kv_layer, void* out, const mk_span_workspace* workspace, int32_t* status_out,
                           mk_stream_t stream);
int mk_prefix_attention_in(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens, const int32_t* seq_lens,
                           int32_t num_groups, const int32_t* group_seqs, const int32_t* prefix_lens,
                           const int32_t* block_tables, const void* q, int64_t q_stride, const void* kv_layer, void* out,
                           const mk_span_workspace* workspace, int32_t* status_out, mk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif
