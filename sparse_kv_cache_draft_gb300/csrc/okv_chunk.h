// Internal declarations of the operators that keep a bounded cache without a context: attention of a chunk of new
// tokens over a paged pool, the weight its slots draw, and eviction by it. Not part of the C ABI.
#pragma once

#include "okv_tree.h"

namespace okv {

struct ChunkArgs {
  Geom G;                     // one layer of G.R requests
  int32_t T;                  // new tokens of a request, at most
  const uint8_t* pool;
  const int32_t* slot_block;
  const int32_t* len;         // tokens before the new ones
  const int32_t* counts;      // [R] new tokens, or NULL: T each
  const void* q;              // [R][T][Hq][d]
  void* out;                  // [R][T][Hq][d]
  float* lse;                 // [R][T][Hq] or NULL
  int32_t window, sinks;      // window: INT32_MAX for none
  const float* weight;        // [R][Hkv][kb] or NULL: zero
  float* weight_out;          // [R][Hkv][kb] or NULL
  int64_t pool_rows;          // slots in `pool`: R * Hkv * kb
};

// Outputs, log sums and, with A.weight_out, what the slots draw.
cudaError_t launch_attend_chunk(const ChunkArgs& A, cudaStream_t s);
// Outputs and log sums of binary32 operands (k_chunk_f32.cu).
cudaError_t launch_chunk_f32(const ChunkArgs& A, cudaStream_t s);
// weight_out = weight + what each slot draws of the rows whose sums are in A.lse.
cudaError_t launch_weigh_chunk(const ChunkArgs& A, cudaStream_t s);

}  // namespace okv
