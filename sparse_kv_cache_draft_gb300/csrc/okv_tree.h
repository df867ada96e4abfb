// Internal declarations of the operators around a decode step: rows of a projection (norm and
// rotation), their append, and attention of a tree of drafted tokens. Not part of the C ABI.
#pragma once

#include "okv_internal.h"

namespace okv {

// The rotation and norms of okv_rotary as the kernels take them.
struct RowArgs {
  int32_t Hq, Hkv, d, half;   // half: rotated pairs of a head
  int32_t interleaved;
  float eps;
  const float* inv_freq;      // [half]
  const void* q_weight;       // [d] or NULL
  const void* k_weight;
  const void* qkv;            // rows of (Hq + 2 Hkv) d elements
  int64_t row_stride;         // elements
  void* q;                    // [rows][Hq][d] or NULL
};

struct TreeArgs {
  Geom G;
  int32_t T;                  // drafted tokens of a request, at most
  const uint8_t* pool;        // one layer's slot pool
  const int32_t* slot_block;
  const int32_t* len;
  const int32_t* active;      // request ids by position, or NULL: 0, 1, ...
  const int32_t* counts;      // [R] drafted tokens, or NULL: T each
  const void *q, *k, *v;      // [R][T][Hq][d], [R][T][Hkv][d] twice
  const uint64_t* mask;       // [R][T]
  void* out;                  // [R][T][Hq][d]
  int64_t pool_rows;          // slots in `pool`: R * Hkv * kb
  Counters* ctr;              // or NULL
  int32_t* err;               // or NULL
};

// Rows 0 .. n - 1: norm and rotation at positions[row] into A.q, k and v (each may be NULL); a row
// with a negative position is left out.
cudaError_t launch_norm_rope(const RowArgs& A, int32_t dtype, int32_t n_rows, const int32_t* positions, void* k, void* v, cudaStream_t s);
// Row r * n_new + t: token t < counts[r] of request r, at position len[r] + t; its key and value go
// into the slot of `pool` that holds its block, if one does.
cudaError_t launch_append_rows(const RowArgs& A, const Geom& G, int32_t n_requests, int32_t n_new, const int32_t* counts, const int32_t* len,
                               const int32_t* slot_block, void* pool, cudaStream_t s);
// One row per active request at its length of `layer`: as launch_append of the normed and rotated
// key and the value, and the query into A.q. Advances the lengths.
cudaError_t launch_append_qkv(const RowArgs& A, const Geom& G, const LayerState& S, const ReqTables& T, int32_t n_active, int32_t layer,
                              int32_t* err, cudaStream_t s);
// The accepted paths of one launch, a kernel parameter: active request first + a appends path[a * stride] drafted
// tokens, those of the bytes behind it, in that order.
struct Accepted {
  int32_t first, stride;
  uint8_t path[3584];  // with the launch's other parameters less than 4 KB
};
// The paths of the n active requests from P.first on.
cudaError_t launch_append_tree(const Geom& G, const LayerState& S, const ReqTables& T, int32_t n, int32_t layer, int32_t n_draft,
                               const void* k, const void* v, const Accepted& P, int32_t* arrivals, int32_t* err, cudaStream_t s);
cudaError_t launch_attend_tree(const TreeArgs& A, int32_t n_active, cudaStream_t s);

// ---- checks of the calls without a context ---------------------------------------------------------
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The limits of okv_create on shapes, as one layer of n_requests requests.
inline bool tree_geom(int32_t n_requests, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t block_size, int32_t slots,
                      int32_t dtype, Geom* out) {
  if (n_requests <= 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || q_heads / kv_heads > 8) return false;
  if (head_dim <= 0 || head_dim % 32 || head_dim > 256 || block_size <= 0 || block_size > 64) return false;
  if (slots <= 0 || slots > 1024 || (dtype != OKV_F32 && dtype != OKV_BF16)) return false;
  // slots, and CTAs of the attention, are counted in 32 bits: a unit has up to 16 groups of rows, whose items are split
  // over further CTAs only where they are fewer than fill the GPU
  if ((int64_t)n_requests * kv_heads * (slots > 16 ? slots : 16) >= ((int64_t)1 << 31)) return false;
  Geom G{};
  G.L = 1;
  G.Hq = q_heads;
  G.Hkv = kv_heads;
  G.g = q_heads / kv_heads;
  G.d = head_dim;
  G.bs = block_size;
  G.kb = slots;
  G.R = n_requests;
  // the blocks of the longest request, the last one part-filled; ids are also checked against each request's length
  G.nb_max = (int32_t)(((int64_t)INT32_MAX + block_size - 1) / block_size);
  G.dtype = dtype;
  G.elem = dtype == OKV_F32 ? 4 : 2;
  G.block_bytes = (int64_t)2 * block_size * head_dim * G.elem;
  *out = G;
  return true;
}

// What a call says of its rows, checked: false if a limit of okv_rotary or of the row layout is not met.
inline bool row_args(const okv_rotary* t, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype, const void* qkv, int64_t row_stride,
                     void* q, RowArgs* out) {
  const int32_t elem = dtype == OKV_F32 ? 4 : 2;
  if (!t || !qkv || !aligned16(qkv) || !aligned16(q)) return false;
  if (q_heads <= 0 || kv_heads <= 0 || q_heads > 4096 || kv_heads > 4096 || q_heads % kv_heads) return false;
  if (head_dim <= 0 || head_dim % 32 || head_dim > 256 || (dtype != OKV_F32 && dtype != OKV_BF16)) return false;
  if (row_stride < (int64_t)(q_heads + 2 * kv_heads) * head_dim || row_stride > INT32_MAX || row_stride * elem % 16) return false;
  if (t->rotary_dim < 0 || t->rotary_dim > head_dim || t->rotary_dim % 16 || (t->rotary_dim && !t->inv_freq)) return false;
  if (!(t->eps >= 0.f) || t->eps > 3.4e38f || !aligned16(t->q_weight) || !aligned16(t->k_weight)) return false;
  if (t->interleaved != 0 && t->interleaved != 1) return false;
  *out = RowArgs{q_heads, kv_heads, head_dim, t->rotary_dim / 2, t->interleaved, t->eps, t->inv_freq, t->q_weight, t->k_weight, qkv, row_stride, q};
  return true;
}

// The kernels run on `stream` on the current device: both must agree. A stream being captured cannot
// be asked for its device (the query would end the capture); there a launch from another device fails
// by itself.
inline okv_status check_stream(void* stream) {
  if (!stream) return OKV_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing((cudaStream_t)stream, &cs) != cudaSuccess) return OKV_ECUDA;
  if (cs != cudaStreamCaptureStatusNone) return OKV_OK;
  int dev = 0, sdev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaStreamGetDevice((cudaStream_t)stream, &sdev) != cudaSuccess) return OKV_ECUDA;
  return sdev == dev ? OKV_OK : OKV_EINVAL;
}

// Lets a launch on s begin while the kernel before it ends (its kernel calls grid_wait): at[0] is filled in and 1
// returned, 0 while s is being captured, where the launches of a graph are plain.
inline int overlap_attr(cudaStream_t s, cudaLaunchAttribute* at) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  return cs == cudaStreamCaptureStatusNone ? 1 : 0;
}

}  // namespace okv
