// The order in which the keys and values of a CTA's tiles use a ring of buffers, and which of their copies may still be on their
// way when a block gives up. For the kernels, and for a host compiler.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define OKV_RING_FN __host__ __device__ __forceinline__
#else
#define OKV_RING_FN inline
#endif

namespace okv {

// Use u takes buffer u % ring, once what use u - ring brought has been read. The uses are in the order in which the MMAs take them. With
// two S buffers, S of tile i + 1 comes before O of tile i: K of tile i is use 2i - 1 (the first: 0), V use 2i + 2. With one, K is
// 2i, V 2i + 1.
template <int kS>
struct RingOrder {
  static OKV_RING_FN int32_t key(int32_t i) { return kS == 1 ? 2 * i : i == 0 ? 0 : 2 * i - 1; }
  static OKV_RING_FN int32_t value(int32_t i) { return kS == 1 ? 2 * i + 1 : 2 * i + 2; }
  // Whether `use` is among those of the keys of tiles 0 .. keys - 1 and the values of tiles 0 .. values - 1.
  static OKV_RING_FN bool among(int32_t use, int32_t keys, int32_t values) {
    if (kS == 1) return use % 2 == 0 ? use / 2 < keys : use / 2 < values;
    return use == 0 ? keys > 0 : use % 2 == 1 ? (use + 1) / 2 < keys : use / 2 - 1 < values;
  }
  // Of the copies that were started, so many of each: whether `use` may be on its way still. One whose buffer was taken again is not: that
  // waited for it to have been read. Only the last of a buffer can be waited for, too: a barrier's parity tells a phase from the next one only.
  static OKV_RING_FN bool may_be_on_its_way(int32_t use, int32_t ring, int32_t keys, int32_t values) { return !among(use + ring, keys, values); }
};

}  // namespace okv
