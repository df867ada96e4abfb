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
// weight_out = weight + what each slot draws of the rows whose sums are in A.lse.
cudaError_t launch_weigh_chunk(const ChunkArgs& A, cudaStream_t s);

// ---- who sees whom --------------------------------------------------------------------------------------
#ifdef __CUDACC__
// New tokens of request r: 0 where its length leaves no room for n_new more positions.
__device__ __forceinline__ int32_t new_tokens(const ChunkArgs& A, int32_t r, int32_t len) {
  if (len < 0 || (int64_t)len + A.T > INT32_MAX) return 0;
  return A.counts ? min(max(A.counts[r], 0), A.T) : A.T;
}

__device__ __forceinline__ uint64_t first_bits(int32_t n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Bits of a slot's bs tokens, the first one at position `base`, that position p sees: those not behind p and less
// than `window` before it, or among the first `sinks`.
__device__ __forceinline__ uint64_t seen_of(int32_t base, int32_t p, int32_t bs, int32_t window, int32_t sinks) {
  if (base > p) return 0;
  const int32_t n = min(bs, p - base + 1), from = max(p - window + 1, 0) - base;
  return (first_bits(n) & ~first_bits(from)) | first_bits(min(sinks - base, n));
}

// What positions p_lo .. p_hi see of block b of bs tokens: 2 all of them every token, 1 some of them some (or, under a
// window with first tokens, perhaps none), 0 nothing.
__device__ __forceinline__ int32_t sight(int32_t b, int32_t bs, int32_t p_lo, int32_t p_hi, int32_t window, int32_t sinks) {
  const int64_t first = (int64_t)b * bs, last = first + bs - 1;
  if (b < 0 || first > p_hi || (last <= (int64_t)p_lo - window && first >= sinks)) return 0;
  return last <= p_lo && (first > (int64_t)p_hi - window || last < sinks) ? 2 : 1;
}
#endif

}  // namespace okv
