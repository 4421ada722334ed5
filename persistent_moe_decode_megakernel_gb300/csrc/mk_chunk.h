// mk_chunk.h -- what the chunk operators' translation units share: the packed sequences of a
// call as kernel parameters, and the checks of the arguments they have in common.
#ifndef MK_CHUNK_INTERNAL_H
#define MK_CHUNK_INTERNAL_H

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mk_chunk.h"

namespace mk {

constexpr int kMaxSeqs = 64;

// The sequences of one call.  They travel as kernel parameters (constant memory), so a call
// uploads nothing and a captured call keeps its own copy.
struct ChunkSeqs {
  int32_t n;                    // sequences
  int32_t row0[kMaxSeqs + 1];   // first packed row of each; row0[n] = rows
  int32_t len[kMaxSeqs];        // length, the new tokens included
};

// The sequence that owns packed row r (0 <= r < row0[n]): the last one that starts at or before
// it and is not empty.
__host__ __device__ inline int seq_of_row(const ChunkSeqs& q, int r) {
  int lo = 0, hi = q.n;         // row0[lo] <= r < row0[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q.row0[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

int chunk_fail(int code, const char* fmt, ...);
// Checks the shape and the lengths and fills `out`; MK_OK or the error (its text set).
int check_chunk(const mk_cache_shape* shape, int32_t num_seqs, const int32_t* chunk_lens, const int32_t* seq_lens,
                ChunkSeqs* out);
// Sets the status word to MK_OK on the stream before a kernel may raise it.
int clear_status(int32_t* status_out, cudaStream_t s);
bool misaligned(const void* p, unsigned bytes);

}  // namespace mk

#endif
