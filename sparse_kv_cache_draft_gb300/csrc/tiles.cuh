// What the attention kernels on the fifth-generation tensor cores share: operand tiles, binary32 products in parts, and how a
// launch covers its items with CTAs and thread-block clusters. Included by the kernels that tile a unit's tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "okv_tree.h"
#include "row_sums.h"
#include "tc5.cuh"

namespace okv {

constexpr int kMaxSplit = 12;     // CTAs of a cluster; above 8 a kernel has to ask for it
constexpr int kMaxSmem = 232448;  // bytes of shared memory a CTA may have

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// Four outputs, one rounding each.
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// How a launch covers its items, (unit, group of rows) with the groups of a unit side by side: clusters of
// `split` CTAs, of which the first take `whole` items, one for each CTA, and the others one item each, dealt
// to their CTAs. So the last items, fewer than would fill the GPU, are shared out.
struct Shape {
  int32_t split, whole, groups;
};

// ---- a cluster's partials -----------------------------------------------------------------------------
// What a CTA hands to its cluster: per row of the group the running maximum (log2 units), sum and
// output (binary32, rows of d with 16-byte chunks at chunk ^ (row & mask)).
struct Partial {
  uint32_t o, m, l;  // shared-memory addresses
};
__device__ __forceinline__ uint32_t part_chunk(int32_t row, int32_t chunk, int32_t d, int32_t xor_mask) {
  return (uint32_t)(row * d * 4 + ((chunk ^ (row & xor_mask)) << 4));
}

// Merges the partials of a cluster's `split` CTAs, this one (`part`) a share of the outputs: finish(row, c, o, M, l) takes
// dims 4 c .. 4 c + 3 of a row, its maximum and its sum. By the first `threads` threads of each CTA, between two cluster_sync that
// every thread of the cluster takes part in.
template <typename F>
__device__ __forceinline__ void merge_rows(int32_t part, int32_t split, int32_t rows, int32_t d, const Partial& P, int32_t xor_mask, int32_t threads,
                                           F finish) {
  const int32_t d4 = d / 4, total = rows * d4;
  for (int32_t i = part * threads + threadIdx.x; i < total; i += split * threads) {
    const int32_t row = i / d4, c = i - row * d4;
    float M = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;  // every load of a batch on its way before the first is used
#pragma unroll 1
    for (int p0 = 0; p0 < split; p0 += kBatch) {
      float m[kBatch], ls[kBatch];
      float4 x[kBatch];
#pragma unroll
      for (int p = 0; p < kBatch; ++p) {
        m[p] = -INFINITY;
        if (p0 + p < split) {
          m[p] = ld_cluster(cluster_map(P.m + row * 4, p0 + p));
          ls[p] = ld_cluster(cluster_map(P.l + row * 4, p0 + p));
          x[p] = ld_cluster4(cluster_map(P.o + part_chunk(row, c, d, xor_mask), p0 + p));
        }
      }
      float mx = M;
#pragma unroll
      for (int p = 0; p < kBatch; ++p) mx = fmaxf(mx, m[p]);
      if (M != -INFINITY) {
        const float f = ex2(M - mx);
        l *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
      }
      M = mx;
#pragma unroll
      for (int p = 0; p < kBatch; ++p) {
        // nothing seen there: its outputs may not have been written. Scores that are all NaN leave no maximum
        // either, but a sum, and the row is then NaN
        if (p0 + p >= split || (m[p] == -INFINITY && ls[p] == 0.f)) continue;
        const float f = ex2(m[p] - M);
        l = fmaf(f, ls[p], l);
        o.x = fmaf(f, x[p].x, o.x);
        o.y = fmaf(f, x[p].y, o.y);
        o.z = fmaf(f, x[p].z, o.z);
        o.w = fmaf(f, x[p].w, o.w);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    finish(row, c, o, M, l);
  }
}

// ---- binary32 products of parts ----------------------------------------------------------------------
struct Parts {
  uint32_t hi, lo;
};
// The tensor cores take the upper 19 bits of an operand as they stand: hi is rounded here, lo is cut off, which
// of a part of either sign leaves no bias.
__device__ __forceinline__ Parts parts_of(float x) {
  const uint32_t hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  return {hi, __float_as_uint(x - __uint_as_float(hi))};
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c[n] += a b[n]. The eight products of a step are summed on the tensor cores, which cut sums off (towards zero);
// the steps are summed here, rounded to nearest. The three products of a sum wait for one another, so the sums take turns.
template <int N>
__device__ __forceinline__ void mma_f32(float (*c)[4], const Parts (&a)[4], const Parts (&b)[N][2]) {
  float x[N][4];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
    mma_tf32(x[n], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[n][0].hi, b[n][1].hi);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) mma_tf32(x[n], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[n][0].lo, b[n][1].lo);
#pragma unroll
  for (int n = 0; n < N; ++n) mma_tf32(x[n], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[n][0].hi, b[n][1].hi);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[n][i] += x[n][i];
}

// ---- operand tiles ------------------------------------------------------------------------------------
// Operand tiles are lines of 64 (or, for d not a multiple of 64, 32) elements: chunk c of a tile is
// [rows][line] under the 128-byte (64-byte) swizzle, Q and K K-major, V MN-major. A K or V tile is d / line
// TMA copies of whole slots, straight from the pool's layout.
template <int D, int Tile>
struct Lines {
  static constexpr int kTile = Tile;                          // tokens of a tile
  static constexpr int kElems = D % 64 == 0 ? 64 : 32;
  static constexpr int kBytes = kElems * 2;
  static constexpr int kChunks = D / kElems;
  static constexpr uint32_t kSwizzle = kElems == 64 ? 2 : 4;  // of the operand descriptors
  static constexpr uint32_t kGroup = 8 * kBytes;              // 8 rows
  static constexpr int kChunk = kTile * kBytes;               // a chunk of a tile
  static constexpr int kBuf = kTile * D * 2;                  // a tile of K or V
  // byte offset of 16-byte piece c (0 .. kBytes / 16 - 1) of line `row` of a chunk
  __device__ static __forceinline__ uint32_t at(int row, int c) {
    return kElems == 64 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
  }
  // ... of 16-byte piece c of token j's line in a tile
  __device__ static __forceinline__ uint32_t piece(int j, int c) {
    return (c / (kBytes / 16)) * kChunk + at(j, c % (kBytes / 16));
  }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// A 16-byte piece of bf16 values with those that are not finite as zero; whether there were any.
__device__ __forceinline__ bool clean(uint4& u) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u, any = true;
    if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu, any = true;
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  return any;
}

// ---- launches -----------------------------------------------------------------------------------------
inline int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

inline cudaLaunchConfig_t cluster_config(int64_t ctas, int threads, size_t smem, int32_t split, cudaStream_t s, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cfg;
}

// Nothing launches it: it stands for kernels of as many threads in the question below (one that allocates tensor
// memory counts as one CTA per SM whatever it allocates).
template <int>
__global__ void room_kernel() {}

// CTAs of clusters of c that run at once, for c = 2 .. 12, where an SM holds per_sm of them: a property of the device
// (a cluster stays within a GPC), asked for once per thread.
struct ClusterRoom {
  int threads, per_sm, dev;
  int64_t ctas[kMaxSplit + 1];
};
inline const ClusterRoom& cluster_room(int threads, int32_t per_sm) {
  constexpr int kKept = 32;
  static thread_local ClusterRoom kept[kKept];
  static thread_local int used = 0, oldest = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  for (int i = 0; i < used; ++i)
    if (kept[i].threads == threads && kept[i].per_sm == per_sm && kept[i].dev == dev) return kept[i];
  ClusterRoom& r = used < kKept ? kept[used++] : kept[oldest++ % kKept];
  r.threads = threads;
  r.per_sm = per_sm;
  r.dev = dev;
  cudaFuncSetAttribute(room_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  cudaFuncSetAttribute(room_kernel<0>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int32_t c = 2; c <= kMaxSplit; ++c) {
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg = cluster_config(c, threads, 233472 / per_sm - 1024, c, nullptr, at);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, room_kernel<0>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    r.ctas[c] = (int64_t)n * c;
  }
  return r;
}

struct Costs {
  double fixed, join, dense;
};
inline double wave_cost(int64_t ctas, double tiles, const Costs& t, int64_t sms) {
  const double crowd = (double)ctas / ((double)sms * t.dense);
  return tiles * (crowd > 1 ? crowd : 1) + t.fixed;
}

// The shape of least cost, of equal ones the one with more CTAs. Items that fill the GPU go whole and the last ones
// split, in pairs: a larger cluster waits behind whole items until all of its CTAs find a place (48 requests of 16
// tokens: 72 us in pairs, 78 whole or in threes; 12 requests: 21 us in threes, 25 in pairs, 29 whole; one of 8 tokens
// 9.2 in twelves, 9.9 in eights, 10.8 in sixteens, which start late; in binary32, one of 4: 19.8, 28.7 and 20.8).
inline Shape pick_shape(int64_t items, int32_t groups, int32_t per_sm, int32_t tiles, const Costs& t, const ClusterRoom& room) {
  const int64_t sms = sm_count(), slots = sms * per_sm;
  const double full = wave_cost(slots, tiles, t, sms);
  Shape best{1, (int32_t)items, groups};
  double least = (double)(items / slots) * full + (items % slots ? wave_cost(items % slots, tiles, t, sms) : 0);
  for (int32_t c = 2; c <= kMaxSplit && c <= tiles; ++c) {
    const int64_t whole = items / slots * slots / c * c, n = (items - whole) * c, r = room.ctas[c];
    if (!r || !n || (whole && c > 2)) continue;
    const double part = (double)tiles / c;
    const double cost = (double)(whole / slots) * full + (double)(n / r) * (wave_cost(r, part, t, sms) + t.join) +
                        (n % r ? wave_cost(n % r, part, t, sms) + t.join : 0);
    if (cost < least + 1e-6) least = cost, best = Shape{c, (int32_t)whole, groups};
  }
  return best;
}

template <typename... P, typename... Q>
cudaError_t launch_cluster(void (*kernel)(P...), int64_t items, const Shape& shape, int threads, size_t smem, cudaStream_t s, Q&&... args) {
  // the limit is the same for every launch: another thread's may come between this and the launch
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess && shape.split > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = cluster_config(shape.whole + (items - shape.whole) * shape.split, threads, smem, shape.split, s, at);
  cfg.numAttrs += overlap_attr(s, at + cfg.numAttrs);
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Q>(args)...);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

}  // namespace okv
