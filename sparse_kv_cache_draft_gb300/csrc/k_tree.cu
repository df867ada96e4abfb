// Attention of a tree of drafted tokens over the resident slot pool.
//
// T <= 64 drafted tokens per request, token i seeing every valid token of the request's occupied
// slots and the drafted tokens whose bit is set in its 64-bit mask. For query head h of KV head k:
//   o_ih = sum_j softmax_j(q_ih . k_j / sqrt(d)) v_j
// over those tokens, zero where there are none (or none has a weight: every score is -infinity). The g T
// rows of a unit (request, KV head) share its keys and values, so a unit's pool is read once for a group of
// rows.
//
// The tokens of a unit are taken in tiles of whole slots (at most 64 tokens, or 128 in bf16 beyond 128 rows);
// tiles without a valid token are left out, the rest are dealt to the CTAs of a thread-block cluster, with the drafted
// tokens as one more tile of the last CTA. Each CTA keeps a running maximum, sum and output per
// row; the cluster merges them through distributed shared memory in rank order, so results do not
// depend on timing and a launch needs no workspace.
//
// Measured (32 / 8 heads of 128 dims, 2048 tokens of context, bf16): 16 tokens x 128 requests 169 us, 6.6
// TB/s, 0.97 of a copy's rate; one request, 8 tokens 9 us. 64 tokens x 32 requests with 64 / 8 heads (512
// rows to a key head) 132 us, 1.04 PFLOP/s, 0.55 of the measured bf16 rate.
#include <cuda_bf16.h>

#include <stddef.h>

#include <utility>

#include "okv_tree.h"
#include "tc5.cuh"

namespace okv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 64;         // tokens of a tile, at most
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

// One CTA's share of the work: a request, a KV head, a group of rows and a part of the tokens.
struct Site {
  int32_t a, r, h, part, parts, cnt, len;  // cnt: drafted tokens of the request
  int32_t row0, rows;                      // rows [row0, row0 + rows) of the unit's g * cnt
  bool first;                              // the first CTA of its unit
};

__device__ __forceinline__ Site make_site(const TreeArgs& A, const Shape& P, int32_t group_rows) {
  Site s;
  const int32_t cluster = blockIdx.x / P.split, rank = blockIdx.x - cluster * P.split, wholes = P.whole / P.split;
  const bool whole = cluster < wholes;
  const int32_t item = whole ? (int32_t)blockIdx.x : P.whole + cluster - wholes;
  const int32_t ua = item / P.groups, group = item - ua * P.groups;
  s.part = whole ? 0 : rank;
  s.parts = whole ? 1 : P.split;
  s.first = group == 0 && s.part == 0;
  s.a = ua / A.G.Hkv;
  s.h = ua - s.a * A.G.Hkv;
  s.r = A.active ? A.active[s.a] : s.a;
  s.cnt = A.counts ? min(max(A.counts[s.r], 0), A.T) : A.T;
  s.len = A.len[s.r];
  s.row0 = group * group_rows;
  s.rows = min(group_rows, s.cnt * A.G.g - s.row0);
  return s;
}
__device__ __forceinline__ uint64_t low_bits(int32_t n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }

// Element offset of row m's vector in q and out, [R][T][Hq][d]; row m is drafted token m / g, head m % g.
__device__ __forceinline__ int64_t row_offset(const TreeArgs& A, const Site& s, int32_t m) {
  const int32_t t = m / A.G.g, j = m - t * A.G.g;
  return (((int64_t)s.r * A.T + t) * A.G.Hq + s.h * A.G.g + j) * A.G.d;
}
// ... and of drafted token t's key and value, [R][T][Hkv][d].
__device__ __forceinline__ int64_t draft_offset(const TreeArgs& A, const Site& s, int32_t t) {
  return (((int64_t)s.r * A.T + t) * A.G.Hkv + s.h) * A.G.d;
}

// The valid tokens of every slot of the unit (0: empty) into nv, and the tiles of spt slots that hold any,
// in order, into `tiles`, with kWhole set where all their places do; their number. One warp. A block id
// outside the request's length counts as an empty slot and is recorded.
constexpr uint32_t kWhole = 0x8000;
struct Slots {
  int32_t b[4];  // of slots lane + 32 u from the first on
};
__device__ __forceinline__ Slots load_slots(const TreeArgs& A, const Site& s, int32_t first) {
  const int32_t* sb = A.slot_block + ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb;
  Slots x;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int32_t i = first + (threadIdx.x & 31) + 32 * u;
    x.b[u] = i < A.G.kb ? sb[i] : -1;
  }
  return x;
}
// `x`: the first slots, loaded ahead.
__device__ __forceinline__ int32_t list_tiles(const TreeArgs& A, const Site& s, Slots x, int32_t spt, uint8_t* nv, uint16_t* tiles) {
  const int lane = threadIdx.x & 31;
  int32_t used = 0;
#pragma unroll 1
  for (int32_t i0 = 0; i0 < A.G.kb; i0 += 128) {
    if (i0) x = load_slots(A, s, i0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int32_t i = i0 + lane + 32 * u, b = x.b[u];
      if (i >= A.G.kb) break;
      int32_t n = 0;
      if (b >= 0) {
        const int64_t rem = (int64_t)s.len - (int64_t)b * A.G.bs;
        if (rem <= 0 || b >= A.G.nb_max) {
          if (A.err) record_error(A.err, kErrBlockRange, -2, s.r, b);
        } else {
          n = (int32_t)(rem < A.G.bs ? rem : A.G.bs);
          ++used;
        }
      }
      nv[i] = (uint8_t)n;
    }
  }
  __syncwarp();
  if (A.ctr && s.first) {
    const int32_t slots = __reduce_add_sync(0xffffffffu, used);
    if (lane == 0) atomicAdd(&A.ctr->attended_slots, (unsigned long long)slots);
  }
  int32_t n = 0;
  for (int32_t t0 = 0; t0 * spt < A.G.kb; t0 += 32) {
    const int32_t first = (t0 + lane) * spt;
    bool any = false, whole = first + spt <= A.G.kb;
    for (int32_t i = first, e = min(first + spt, A.G.kb); i < e; ++i) {
      any = any || nv[i];
      whole = whole && nv[i] == A.G.bs;
    }
    const unsigned have = __ballot_sync(0xffffffffu, any);
    if (any) tiles[n + __popc(have & ((1u << lane) - 1u))] = (uint16_t)(t0 + lane | (whole ? kWhole : 0u));
    n += __popc(have);
  }
  return n;
}
__device__ __forceinline__ int32_t tile_of(uint16_t t) { return t & (kWhole - 1); }

// Adds what the drafted values that are not finite give to four outputs (dims c .. c + 3) of a row
// that sees them. Those elements are zero in the products, where a weight of zero times them would
// reach rows that do not see them.
template <typename T>
__device__ __forceinline__ void add_not_finite(const TreeArgs& A, const Site& s, uint64_t seen, int32_t c, float4& o) {
  while (seen) {
    const int32_t t = __ffsll((long long)seen) - 1;
    seen &= seen - 1;
    const T* v = (const T*)A.v + draft_offset(A, s, t) + c;
    const float x = to_f(v[0]), y = to_f(v[1]), z = to_f(v[2]), w = to_f(v[3]);
    if (!is_finite(x)) o.x += x;
    if (!is_finite(y)) o.y += y;
    if (!is_finite(z)) o.z += z;
    if (!is_finite(w)) o.w += w;
  }
}

// What a CTA hands to its cluster: per row of the group the running maximum (log2 units), sum and
// output (binary32, rows of d with 16-byte chunks at chunk ^ (row & mask)).
struct Partial {
  uint32_t o, m, l, bad;  // shared-memory addresses; bad: the drafted values that are not finite
};
__device__ __forceinline__ uint32_t part_chunk(int32_t row, int32_t chunk, int32_t d, int32_t xor_mask) {
  return (uint32_t)(row * d * 4 + ((chunk ^ (row & xor_mask)) << 4));
}

// Merges the cluster's partials, each CTA a share of the outputs, and writes them. Every thread of
// every CTA of the cluster calls it.
template <typename T>
__device__ __forceinline__ void merge_cluster(const TreeArgs& A, const Site& s, const Partial& P, int32_t xor_mask) {
  const int32_t split = s.parts;
  cluster_sync();
  const int32_t d4 = A.G.d / 4, total = s.rows * d4;
  const uint64_t bad = ld_cluster_u64(cluster_map(P.bad, split - 1));
  for (int32_t i = s.part * blockDim.x + threadIdx.x; i < total; i += split * blockDim.x) {
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
          x[p] = ld_cluster4(cluster_map(P.o + part_chunk(row, c, A.G.d, xor_mask), p0 + p));
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
    const int32_t mrow = s.row0 + row;
    if (bad) add_not_finite<T>(A, s, bad & A.mask[(int64_t)s.r * A.T + mrow / A.G.g], c * 4, o);
    store4((T*)A.out + row_offset(A, s, mrow) + c * 4, o);
  }
  cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// ---- binary32 ------------------------------------------------------------------------------------------
//
// Products of binary32 numbers on the tensor cores, as three products of 11-bit parts: x = hi + lo + less
// than 2^-21 x, hi the upper 11 bits and lo the next 11, and x y = hi hi + hi lo + lo hi within 2^-20 of
// |x y|; sums in binary32. (On the CUDA cores the reads of shared memory bound both products: 25 TFLOP/s at
// 64 tokens x 16 requests, 32 / 8 heads, d 128, 2048 tokens of context.) The parts of an operand that is not finite, or
// within 2^-12 of the largest number, do not add up to it: a score is then NaN (hi and lo are infinities of both signs) and
// its weight with it, an output NaN or infinite, and neither a row's sum of weights nor an output becomes finite again. So a
// CTA that ends with one that is not finite takes its tiles again, those scores and all outputs by plain products.
//
// 128 threads, 16 RG rows x 64 tokens; a warp takes 16 rows and 64 / TH of the tokens with a maximum, sum and
// output of its own, merged at the end. m16n8k8: S's accumulators are P's operand as they stand, with the
// tokens 2t and 2t + 1 of a lane as k = t and t + 4, and V's rows read in that order. Rows of d + 4 floats
// keep all fragment reads free of bank conflicts. Tokens are copied whole, by bulk copies that zeros stand in for
// where a token is not valid (by 16-byte pieces the issue of a tile's copies took as long as its scores).
// 12 tokens x 16 requests, 8 / 2 heads of 64 dims, 512 tokens of context: 18.7 us against 36 on the CUDA cores;
// 35 TFLOP/s at the shape above (30 before the bulk copies and before the three products took turns), 105 of the
// 301 that these MMAs alone reach: bound by the splitting of the operands and the reads of shared memory, about
// 15 instructions to 3 MMAs, at 8 warps on an SM.
constexpr int kF32Threads = 128;

__host__ __device__ constexpr int f32_pitch(int d) { return d + 4; }
__host__ __device__ constexpr size_t f32_smem(int d, int rg, int kb, int tiles) {
  const int th = 4 / rg;
  return (size_t)(16 * rg + 2 * kTile) * f32_pitch(d) * 4 + (size_t)(th + 1) * 16 * rg * 8 + 48 + ((size_t)kb + 15) / 16 * 16 + (size_t)tiles * 2;
}
__host__ __device__ constexpr int f32_ctas(int dv) { return dv <= 4 ? 3 : 2; }  // CTAs of an SM, by registers

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

template <int DV, int RG>
__global__ void __launch_bounds__(kF32Threads, f32_ctas(DV)) tree_f32_kernel(const TreeArgs A, const Shape shape) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int d = DV * 32, pitch = f32_pitch(d), kRows = 16 * RG, TH = 4 / RG, kTok = kTile / TH, NT = kTok / 8;
  float* qs = reinterpret_cast<float*>(smem);      // [rows][pitch]
  float* ks = qs + kRows * pitch;                  // [64][pitch]
  float* vs = ks + kTile * pitch;                  // [64][pitch]
  float* ms = vs + kTile * pitch;                  // [rows], then [TH][rows] of the warps
  float* ls = ms + (TH + 1) * kRows;               // the same
  uint64_t* bad = reinterpret_cast<uint64_t*>(ls + (TH + 1) * kRows);
  uint64_t* bars = bad + 1;                        // keys, values, queries there
  int32_t* n_tiles = reinterpret_cast<int32_t*>(bars + 3);
  uint8_t* nv = reinterpret_cast<uint8_t*>(n_tiles + 4);
  uint16_t* tiles = reinterpret_cast<uint16_t*>(nv + (A.G.kb + 15) / 16 * 16);

  if (threadIdx.x == 0) {
    *bad = 0;
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(bars + i), i < 2 ? kTile : kRows);
    fence_mbar_init();
    fence_proxy_async();
  }
  __syncthreads();
  grid_wait();
  grid_go();
  const Site s = make_site(A, shape, kRows);
  if (s.rows <= 0) return;
  const int32_t split = s.parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, ti = lane & 3;
  const int rg = warp % RG, th = warp / RG, tok0 = th * kTok;
  const int32_t bs = A.G.bs, spt = kTile / bs, tt = spt * bs;
  constexpr int kPieces = d / 4, kEach = kTile * kPieces / kF32Threads;  // 16-byte pieces of a token, of a thread's share of a tile
  // Rows are copied whole, each by a thread that counts it at the barrier of its tile.
  auto copy_row = [&](uint32_t bar, float* to, const float* from) {
    mbar_expect_tx(bar, d * 4);
    bulk_load(smem_u32(to), from, d * 4, bar);
  };
  if (tid >= 64 && tid < 64 + kRows) {
    const int row = tid - 64;  // rows past the group's are never read out
    if (row < s.rows)
      copy_row(smem_u32(bars + 2), qs + row * pitch, (const float*)A.q + row_offset(A, s, s.row0 + row));
    else
      mbar_arrive(smem_u32(bars + 2));
  }
  if (tid < 32) {
    const int32_t n = list_tiles(A, s, load_slots(A, s, 0), spt, nv, tiles);
    if (tid == 0) *n_tiles = n;
  }
  __syncthreads();
  const bool draft = s.part == split - 1;
  const int32_t mine = (*n_tiles - s.part + split - 1) / split + (draft ? 1 : 0);
  const float scale = kLog2e / sqrtf((float)d);
  const uint8_t* unit = A.pool + ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb * A.G.block_bytes;
  const uint32_t per_bs = (65536 + bs - 1) / bs;  // j * per_bs >> 16 is j / bs for j < 64
  auto entry = [&](int32_t it) { return tiles[s.part + (it - (draft ? 1 : 0)) * split]; };
  // Tile it's keys (which = 0) or values into shared memory, by 64 threads, a token each. A value that is no
  // valid token's is zero, as its weight of zero needs; a key may be anything.
  auto load = [&](int32_t it, int which) {
    if (it >= mine) return;
    const int32_t j = tid & 63;
    const float* from = nullptr;
    if (draft && it == 0) {
      if (j < s.cnt) from = (const float*)(which ? A.v : A.k) + draft_offset(A, s, j);
    } else {
      const int32_t in = j * per_bs >> 16, slot = tile_of(entry(it)) * spt + in, off = j - in * bs;
      if (j < tt && slot < A.G.kb && off < nv[slot])
        from = reinterpret_cast<const float*>(unit + slot * A.G.block_bytes) + (int64_t)(which * bs + off) * d;
    }
    const uint32_t bar = smem_u32(bars + which);
    float* to = (which ? vs : ks) + j * pitch;
    if (from) {
      copy_row(bar, to, from);
    } else {
      if (which)
        for (int c = 0; c < d; c += 4) *reinterpret_cast<float4*>(to + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      mbar_arrive(bar);
    }
  };
  load(0, tid >> 6);

  uint64_t sees[2];  // of rows gi and gi + 8 of the warp's 16
  bool real[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t row = rg * 16 + gi + 8 * i;
    real[i] = row < s.rows;
    sees[i] = real[i] ? A.mask[(int64_t)s.r * A.T + (s.row0 + row) / A.G.g] & low_bits(s.cnt) : 0;
  }
  float o[d / 8][4], m[2], l[2];
  bool ok = mbar_wait_timed(smem_u32(bars + 2), 0), failed = false, again = false;
  auto phase = [&](int32_t it) { return (uint32_t)((again ? mine + it : it) & 1); };
  for (;; again = true) {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < d / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    for (int32_t it = 0; it < mine && !failed; ++it) {
      const bool is_draft = draft && it == 0;
      uint64_t vis[2] = {sees[0], sees[1]};
      if (!is_draft) {
        const uint16_t tile = entry(it);
        uint32_t half[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int32_t j = lane + 32 * u, in = j * per_bs >> 16, slot = tile_of(tile) * spt + in;
          half[u] = __ballot_sync(0xffffffffu, j < tt && slot < A.G.kb && j - in * bs < nv[min(slot, A.G.kb - 1)]);
        }
        vis[0] = real[0] ? (uint64_t)half[1] << 32 | half[0] : 0;
        vis[1] = real[1] ? (uint64_t)half[1] << 32 | half[0] : 0;
      }
      ok = mbar_wait_timed(smem_u32(bars), phase(it)) && ok;
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
      const float* qa = qs + (rg * 16 + gi) * pitch + ti;
      const float* kr = ks + (tok0 + gi) * pitch + ti;
#pragma unroll 4
      for (int k = 0; k < d; k += 8) {
        const Parts a[4] = {parts_of(qa[k]), parts_of(qa[k + 8 * pitch]), parts_of(qa[k + 4]), parts_of(qa[k + 8 * pitch + 4])};
        Parts b[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n][0] = parts_of(kr[n * 8 * pitch + k]), b[n][1] = parts_of(kr[n * 8 * pitch + k + 4]);
        mma_f32<NT>(sc, a, b);
      }
      // rows gi: sc[.][0], sc[.][1]; gi + 8: sc[.][2], sc[.][3]; tokens tok0 + 8 n + 2 ti and the next
      if (again) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (is_finite(sc[n][e])) continue;
            const float *x = qs + (rg * 16 + gi + 8 * (e >> 1)) * pitch, *y = ks + (tok0 + 8 * n + 2 * ti + (e & 1)) * pitch;
            float sum = 0.f;
#pragma unroll 1
            for (int k = 0; k < d; ++k) sum = fmaf(x[k], y[k], sum);
            sc[n][e] = sum;
          }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = sc[n][2 * i + e];
            x = vis[i] >> (tok0 + 8 * n + 2 * ti + e) & 1 ? x * scale : -INFINITY;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn, f = ex2(m[i] - ref);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) sum += sc[n][2 * i + e] = ex2(sc[n][2 * i + e] - ref);
        l[i] = l[i] * f + sum;  // of this lane's tokens; summed over the four lanes at the end
#pragma unroll
        for (int n = 0; n < d / 8; ++n) {
          o[n][2 * i] *= f;
          o[n][2 * i + 1] *= f;
        }
      }
      __syncthreads();
      if (tid < 64) load(it + 1, 0);  // the keys have been read
      ok = mbar_wait_timed(smem_u32(bars + 1), phase(it)) && ok;
      if (is_draft) {
        // values that are not finite are zero in the products
#pragma unroll 1
        for (int u = 0; u < kEach; ++u) {
          const int i = tid + u * kF32Threads, j = i / kPieces, c = i % kPieces;
          float4* at = reinterpret_cast<float4*>(vs + j * pitch + c * 4);
          float4 y = *at;
          if (is_finite(y.x) && is_finite(y.y) && is_finite(y.z) && is_finite(y.w)) continue;
          atomicOr(reinterpret_cast<unsigned long long*>(bad), 1ull << j);
          if (!is_finite(y.x)) y.x = 0.f;
          if (!is_finite(y.y)) y.y = 0.f;
          if (!is_finite(y.z)) y.z = 0.f;
          if (!is_finite(y.w)) y.w = 0.f;
          *at = y;
        }
        __syncthreads();
      }
      if (!again) {
        const float* vr = vs + (tok0 + 2 * ti) * pitch + gi;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const Parts a[4] = {parts_of(sc[n][0]), parts_of(sc[n][2]), parts_of(sc[n][1]), parts_of(sc[n][3])};
#pragma unroll
          for (int c = 0; c < d / 8; c += 4) {
            Parts b[4][2];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              b[e][0] = parts_of(vr[n * 8 * pitch + (c + e) * 8]), b[e][1] = parts_of(vr[n * 8 * pitch + pitch + (c + e) * 8]);
            mma_f32<4>(o + c, a, b);
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {  // token 8 n + 2 u + e, whose weights are with lane u of the row
              const float p = __shfl_sync(0xffffffffu, sc[n][e], (lane & 28) | u), p8 = __shfl_sync(0xffffffffu, sc[n][2 + e], (lane & 28) | u);
              const float* v = vs + (tok0 + 8 * n + 2 * u + e) * pitch + 2 * ti;
#pragma unroll
              for (int c = 0; c < d / 8; ++c) {
                const float2 y = *reinterpret_cast<const float2*>(v + c * 8);
                o[c][0] = fmaf(p, y.x, o[c][0]);
                o[c][1] = fmaf(p, y.y, o[c][1]);
                o[c][2] = fmaf(p8, y.x, o[c][2]);
                o[c][3] = fmaf(p8, y.y, o[c][3]);
              }
            }
      }
      failed = __syncthreads_or(!ok) != 0;
      if (tid >= 64 && !failed) {  // the values have been read
        fence_proxy_async();       // zeros were written among them
        load(it + 1, 1);
      }
      if (failed && it + 1 < mine) mbar_wait_timed(smem_u32(bars), phase(it + 1));  // copies in flight land (bounded)
    }
    bool odd = real[0] && !is_finite(l[0]) || real[1] && !is_finite(l[1]);
#pragma unroll
    for (int n = 0; n < d / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) odd |= real[e >> 1] && !is_finite(o[n][e]);
    if (again || failed || !__syncthreads_or(odd)) break;
    fence_proxy_async();
    load(0, tid >> 6);
  }
  if (failed || !ok) {  // a row of a CTA that gave up has seen nothing
    if (A.err && tid == 0) record_error(A.err, kErrTimeout, -3, s.r, 6);
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < d / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  }
  __syncthreads();  // every tile read: keys and values give way to the warps' outputs, [TH][rows][d]
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const int row = rg * 16 + gi + 8 * i;
    float* to = ks + (th * kRows + row) * d + 2 * ti;
#pragma unroll
    for (int c = 0; c < d / 8; ++c) *reinterpret_cast<float2*>(to + c * 8) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
    if (ti == 0) {
      ms[(1 + th) * kRows + row] = m[i];
      ls[(1 + th) * kRows + row] = l[i];
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < s.rows * kPieces; i += kF32Threads) {
    const int row = i / kPieces, c = i % kPieces;
    float M = -INFINITY, sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 1; k <= TH; ++k) M = fmaxf(M, ms[k * kRows + row]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int k = 0; k < TH; ++k) {
      const float f = ex2(ms[(1 + k) * kRows + row] - ref);
      const float4 y = *reinterpret_cast<const float4*>(ks + (k * kRows + row) * d + c * 4);
      sum = fmaf(f, ls[(1 + k) * kRows + row], sum);
      x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
    }
    if (split > 1) {
      *reinterpret_cast<float4*>(ks + row * d + c * 4) = x;  // read above by this thread alone
      if (c == 0) {
        ms[row] = M;
        ls[row] = sum;
      }
      continue;
    }
    const float inv = 1.f / sum;
    x = sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    const int32_t mrow = s.row0 + row;
    if (*bad) add_not_finite<float>(A, s, *bad & A.mask[(int64_t)s.r * A.T + mrow / A.G.g], c * 4, x);
    store4((float*)A.out + row_offset(A, s, mrow) + c * 4, x);
  }
  if (split > 1) merge_cluster<float>(A, s, Partial{smem_u32(ks), smem_u32(ms), smem_u32(ls), smem_u32(bad)}, 0);
}

// ---- tensor cores: bf16 ------------------------------------------------------------------------------
//
// A CTA holds NW groups of 128 rows (one softmax warpgroup each) over the same tiles of tokens. One warp
// copies K and V tiles by TMA into a ring of buffers, a warp for each group issues its MMAs:
//   S = Q K^T   128 x tile, Q and K in shared memory, S in TMEM
//   O += P V    128 x d,    P in TMEM in the place of its S (bf16), V in shared memory, O in TMEM
// and a thread of the warpgroup takes a row's softmax.
//
// Up to 128 rows (NW = 1) HBM is the limit: tiles are 64 tokens, two CTAs share an SM, and S has two
// buffers, so that S of the next tile is there before this one's softmax is done. Beyond (NW = 2) it is the
// tensor cores: tiles are 128 tokens (an MMA of 64 columns takes no less time for its A than one of 128)
// and one S buffer per warpgroup is enough, as each warpgroup's softmax runs beside the other's products.
// The running maximum moves only when a row grows past it by 2^8 (the weights then stay below 2^8,
// exact in binary32 sums and as exact in bf16 as any other); only then is O read back and scaled.
// Weights are rounded to bf16 for the second product, as the tensor cores take them; their sum is of
// the unrounded weights.
//
// What bounds it. Up to 128 rows, HBM, but for the CTAs' starts and ends, which the other CTA of the SM
// covers: 4 us of the 168 are above the bytes' time. Beyond, the chain of one warpgroup: 128 scores of a row
// in a thread take about 1500 cycles, O and the next S 1100 more and 400 to pass between them, twice in turn
// where the tensor cores alone would need 2050. The steps that counted, 16 tokens x 128 requests / 64 tokens x
// 32 requests: first version 217 / 286 us; MMAs issued by a whole warp, so that descriptors are in uniform
// registers, 186 / 227; tiles of 128 tokens beyond 128 rows - / 204; queries and drafted tokens by TMA, outputs
// through shared memory - / 182; the last items split, 180 / 165; the running maximum of a warp's rows moved
// together 173 / 156; turns at the tensor cores - / 140; barriers and slot table set up before the lengths are
// there 171 / 134; launches that overlap 168 / 132. Slower: weights taken against the old maximum and again where it moved (208), scores in
// sets of 32 (151), S of 64 tokens in two buffers beyond 128 rows (152); no faster: one S for both warpgroups in
// turn with a P of their own, P in halves (132).
//
// Rows past the group's are whatever the shared memory behind Q holds: they reach only outputs that
// are not stored, have no vote on the running maxima, and warps of such rows skip the softmax.
//
// Operand tiles are lines of 64 (or, for d not a multiple of 64, 32) elements: chunk c of a tile is
// [rows][line] under the 128-byte (64-byte) swizzle, Q and K K-major, V MN-major. A K or V tile is d / line
// TMA copies of whole slots, straight from the pool's layout.

template <int D, int NW>
struct Lines {
  static constexpr int kTile = NW == 2 ? 128 : 64;            // tokens of a tile
  static constexpr int kS = 128 / kTile;                      // S buffers
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

// S, P and O have a barrier each for even and for odd tiles: a barrier's parity tells a phase from the next
// one only, and with two S buffers the softmax may be done with tile i + 1 before the issuing warp has
// looked at tile i, as that warp may be done with O of tile i - 1 before the softmax has looked at tile i - 2.
constexpr int kMaxRing = 12;
struct MmaBars {
  uint64_t full[kMaxRing], empty[kMaxRing], q_full, s_full[2][2], p_full[2][2], pv_done[2][2], drain[2], turn[2];
  uint64_t bad, bad_of[8];  // drafted tokens with values that are not finite: all, found by each warp
  uint32_t tmem;
  int32_t n_tiles, failed;
};

__host__ __device__ constexpr size_t mma_misc(int kb, int tiles) {
  return sizeof(MmaBars) + ((size_t)kb + 15) / 16 * 16 + (size_t)tiles * 2;
}

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

// The tensor maps of a launch: the pool, the queries and the drafted keys and values.
struct MmaMaps {
  CUtensorMap pool, q, k, v;
};

template <int D, int NW>
__global__ void __launch_bounds__(NW * 160 + 32, D <= 128 && NW == 1 ? 2 : 1)
tree_mma_kernel(const TreeArgs A, const __grid_constant__ MmaMaps M, const Shape shape, const int32_t ring, const int32_t q_tok, const int32_t q_rows) {
  using L = Lines<D, NW>;
  constexpr int kTile = L::kTile, kS = L::kS;
  constexpr uint32_t kCols = D <= 128 ? 256 : 512;  // TMEM columns of a warpgroup: S in the first 128, O behind
  constexpr uint32_t kO = 128;
  constexpr uint32_t kDescQK = mma_desc_bf16(128, kTile, false), kDescPV = mma_desc_bf16(128, D, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem;                                                        // [NW][chunks][q_rows][line]
  uint8_t* rs = qs + (size_t)NW * q_rows * D * 2;                            // [ring][chunks][tile][line]
  MmaBars& B = *reinterpret_cast<MmaBars*>(rs + (size_t)ring * L::kBuf);
  uint8_t* nv = reinterpret_cast<uint8_t*>(&B + 1);                          // [kb]
  uint16_t* tiles = reinterpret_cast<uint16_t*>(nv + (A.G.kb + 15) / 16 * 16);

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool is_copy = warp == NW * 4, is_mma = warp > NW * 4;
  const int32_t gr = q_tok * A.G.g;  // rows of a warpgroup: q_tok drafted tokens, all heads of the group
  if (is_copy) {  // what reads no memory of the call
    if (lane < 4) tma_prefetch_map(&M.pool + lane);
    // the barriers, one to a lane: a buffer is free when every warpgroup's product has read it
    constexpr int kEmpty = offsetof(MmaBars, empty) / 8, kP = offsetof(MmaBars, p_full) / 8;
    for (int i = lane; i < (int)(offsetof(MmaBars, bad) / 8); i += 32)
      mbar_init(smem_u32(B.full + i), i >= kEmpty && i < kEmpty + kMaxRing ? NW : i >= kP && i < kP + 4 ? 128 : 1);
  }
  grid_wait();
  const Site s = make_site(A, shape, NW * gr);
  Slots first_slots;
  if (is_copy) first_slots = load_slots(A, s, 0);  // needs no length yet, while that is on its way
  if (s.rows <= 0) return;
  const int32_t split = s.parts;
  const bool draft = s.part == split - 1;  // this CTA's tile 0 is the drafted tokens
  const int32_t bs = A.G.bs, spt = kTile / bs, tt = spt * bs;
  const uint32_t ring0 = smem_u32(rs);

  // The uses of the ring are in the order in which the MMAs take them. With two S buffers, S of tile i + 1
  // comes before O of tile i: K of tile i is use 2i - 1 (the first: 0), V use 2i + 2. With one, K is 2i, V 2i + 1.
  auto v_use = [](int32_t i) { return kS == 2 ? 2 * i + 2 : 2 * i + 1; };
  auto uses = [](int32_t tiles_) { return kS == 2 ? 2 * tiles_ + 1 : 2 * tiles_; };
  auto full = [&](int32_t use) { return mbar_wait_timed(smem_u32(&B.full[use % ring]), (uint32_t)((use / ring) & 1)); };
  // ... by all lanes of a warp: what follows is by whole warps
  auto warp_wait = [&](uint64_t& bar, int32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_timed(smem_u32(&bar), (uint32_t)parity)) != 0;
  };
  auto fail = [&](int32_t site) {
    *(volatile int32_t*)&B.failed = 1;
    if (A.err) record_error(A.err, kErrTimeout, -3, s.r, site);
  };
  const int32_t lead = draft ? 1 : 0;
  int32_t n = 0;          // this CTA's tiles
  // copy warp: the next use to fill, its buffer and the parity of its fill
  int32_t next = 0, next_buf = 0, next_par = 0, issued = 0;
  const int32_t unit_slot = (int32_t)(((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb);
  auto fill = [&] {
    const int32_t use = next, b = next_buf, parity = next_par;
    const bool v = kS == 2 ? use > 0 && use % 2 == 0 : use % 2 == 1;
    const int32_t i = kS == 1 ? use / 2 : v ? use / 2 - 1 : (use + 1) / 2;
    ++next;
    if (++next_buf == ring) next_buf = 0, next_par ^= 1;
    if (i < lead || i >= n) return true;  // the drafted tokens, or the use that a further K would have
    if (use >= ring && !mbar_wait_timed(smem_u32(&B.empty[b]), (uint32_t)(parity ^ 1))) return false;
    const uint32_t bar = smem_u32(&B.full[b]);
    const int32_t slot = unit_slot + tile_of(tiles[s.part + (i - lead) * split]) * spt;
    mbar_expect_tx(bar, (uint32_t)(tt * D * 2));
#pragma unroll
    for (int c = 0; c < L::kChunks; ++c) tma_load_5d(ring0 + b * L::kBuf + c * L::kChunk, &M.pool, bar, 0, c, 0, v ? 1 : 0, slot);
    issued = next;
    return true;
  };

  // Setup: the copy warp starts the copies of the queries and the drafted tokens, reads the slot table and
  // starts the pool's copies that need no free buffer.
  if (is_copy) {
    fence_mbar_init();
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      B.failed = 0;
      // rows (t, head of the group) of a box follow one another as the group's rows do; a box past the last
      // request's tokens is filled up with zeros
      const uint32_t q_bar = smem_u32(&B.q_full);
      const int32_t boxes = NW > 1 && s.rows > gr ? 2 : 1, tok0 = s.r * A.T;
      mbar_expect_tx(q_bar, (uint32_t)(boxes * gr * D * 2));
      for (int w = 0; w < boxes; ++w)
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_5d(smem_u32(qs) + (w * L::kChunks + c) * q_rows * L::kBytes, &M.q, q_bar, 0, c, 0, s.h, tok0 + s.row0 / A.G.g + w * q_tok);
      if (draft)
        for (int e = 0; e < 2; ++e) {
          const int32_t b = e ? v_use(0) : 0;
          const uint32_t bar = smem_u32(&B.full[b]);
          mbar_expect_tx(bar, (uint32_t)(A.T * D * 2));
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_5d(ring0 + b * L::kBuf + c * L::kChunk, e ? &M.v : &M.k, bar, 0, c, s.h, tok0, 0);
        }
    }
    __syncwarp();
    const int32_t all = list_tiles(A, s, first_slots, spt, nv, tiles);
    __syncwarp();
    n = (all - s.part + split - 1) / split + lead;
    if (lane == 0) {
      B.n_tiles = n;
      while (next < 2 && next < uses(n)) fill();  // the others behind the barrier below
    }
  } else if (is_mma) {
    if (warp == NW * 4 + 1) tmem_alloc(smem_u32(&B.tmem), kCols * NW);
  } else {
    uint64_t bad = 0;
    if (draft) {
      // the lines behind the drafted tokens' values meet weights of zero
      constexpr int kPieces = D / 8;
#pragma unroll 1
      for (int e = A.T * kPieces + tid; e < kTile * kPieces; e += NW * 128)
        *reinterpret_cast<uint4*>(rs + v_use(0) * L::kBuf + L::piece(e / kPieces, e % kPieces)) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
      // are there values that are not finite?
#pragma unroll 1
      for (int e0 = tid; e0 < s.cnt * kPieces; e0 += 4 * NW * 128) {
        uint4 y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u * NW * 128;
          y[u] = make_uint4(0, 0, 0, 0);
          if (e < s.cnt * kPieces) y[u] = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)A.v + draft_offset(A, s, e / kPieces) + e % kPieces * 8);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (clean(y[u])) bad |= 1ull << (e0 + u * NW * 128) / kPieces;
      }
      bad = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(bad >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)bad);
    }
    if (lane == 0) B.bad_of[warp] = bad;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_go();  // the TMEM is allocated
  const uint32_t tmem = __shfl_sync(0xffffffffu, B.tmem, 0);
  n = __shfl_sync(0xffffffffu, B.n_tiles, 0);
  if (tid == 0) {
    uint64_t bad = 0;
    for (int i = 0; i < NW * 4; ++i) bad |= B.bad_of[i];
    B.bad = bad;  // read behind the loops
  }
  float m_run = -INFINITY, l_run = 0.f;

  if (is_copy) {
    if (lane == 0) {
      bool ok = true;
      while (next < uses(n) && ok) ok = fill();
      if (!ok) {
        fail(0);
        // the copies still in flight land before the shared memory is given up (bounded)
        for (int32_t use = issued > ring ? issued - ring : 0; use < issued; ++use) full(use);
        if (draft && issued <= ring) full(0), full(v_use(0));
      }
      if (!ok || n == 0) mbar_wait_timed(smem_u32(&B.q_full), 0);  // else the MMA warp has seen it
    }
  } else if (is_mma) {
    const bool one = lane == 0;
    constexpr int kSteps = L::kElems / 16;
    constexpr uint32_t kHi = smem_desc_hi(L::kGroup, L::kSwizzle);
    const int w = warp - NW * 4 - 1;  // the warpgroup it works for
    const uint32_t my = tmem + w * kCols;
    const uint32_t q_chunk = (uint32_t)(q_rows * L::kBytes) >> 4;
    const uint32_t q_desc = smem_desc_lo(smem_u32(qs), 16) + w * L::kChunks * q_chunk, k_desc = smem_desc_lo(ring0, 16);
    const uint32_t v_desc = smem_desc_lo(ring0, L::kChunk);
    int32_t kb = 0, kp = 0, vb = v_use(0), vp = 0;  // buffers and parities of the next K and V
    auto step = [&](int32_t& b, int32_t& parity, int32_t by) {
      b += by;
      if (b >= ring) b -= ring, parity ^= 1;
    };
    auto k_ready = [&] {
      if (!warp_wait(B.full[kb], kp)) return false;
      tc_fence_after();
      return true;
    };
    auto qk = [&](int32_t i) {
      const uint32_t kd = k_desc + kb * (L::kBuf >> 4);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        mma_ss(my + (kS == 2 ? (i & 1) * kTile : 0), q_desc + c / kSteps * q_chunk + c % kSteps * 2, kd + c / kSteps * (L::kChunk >> 4) + c % kSteps * 2,
               kHi, kDescQK, c > 0, one);
      mma_commit(smem_u32(&B.s_full[w][i & 1]), one);
      mma_commit(smem_u32(&B.empty[kb]), one);
      step(kb, kp, kS == 2 && i == 0 ? 1 : 2);
    };
    // Two warpgroups take turns at the tensor cores, O of a tile and S of the next at a time: while one has
    // them, the other is at its softmax. Left to themselves they end up side by side, waiting for each other
    // at both (64 tokens x 32 requests, 64 / 8 heads, d 128, 2048 tokens of context: 153 us
    // against 144).
    int32_t turns = 0;
    auto my_turn = [&] { return NW == 1 || (w == 0 && turns == 0) || warp_wait(B.turn[w], (turns - (w == 0)) & 1); };
    auto pass_on = [&] {
      ++turns;
      if (NW == 2 && one) mbar_arrive(smem_u32(&B.turn[w ^ 1]));
    };
    bool ok = true;
    if (n > 0) {
      ok = warp_wait(B.q_full, 0) && k_ready() && my_turn();
      if (ok) qk(0);
      pass_on();
    }
    for (int32_t i = 0; i < n && ok; ++i) {
      if (i + 1 < n) ok = k_ready();
      if (kS == 2 && ok && i + 1 < n) qk(i + 1);
      ok = ok && warp_wait(B.full[vb], vp) && my_turn() && warp_wait(B.p_full[w][i & 1], (i >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t vd = v_desc + vb * (L::kBuf >> 4);
#pragma unroll
      for (int c = 0; c < kTile / 16; ++c)
        mma_ts(my + kO, my + (kS == 2 ? (i & 1) * kTile : 0) + c * 8, vd + c * 2 * (L::kGroup >> 4), kHi, kDescPV,
               i > 0 || c > 0, one);
      mma_commit(smem_u32(&B.pv_done[w][i & 1]), one);
      mma_commit(smem_u32(&B.empty[vb]), one);
      step(vb, vp, 2);
      if (kS == 1 && i + 1 < n) qk(i + 1);  // S takes the place of the P just used: the products run in order
      pass_on();
    }
    if (!ok) {
      fail(1);
      mma_commit(smem_u32(&B.drain[w]), one);
      warp_wait(B.drain[w], 0);
    }
  } else {
    const int w = warp >> 2, row = tid & 127, wrow = w * gr + row;
    const bool real = row < gr && wrow < s.rows, active = (warp & 3) * 32 < min(gr, s.rows - w * gr);
    const uint32_t my = tmem + w * kCols + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the TMEM lanes
    const float scale = kLog2e * rsqrtf((float)D);
    uint64_t sees = 0, bad = 0;
    for (int k = 0; k < NW * 4; ++k) bad |= B.bad_of[k];
    if (!real) m_run = INFINITY;  // no vote below: what such a row holds moves no other row's maximum
    if (draft && real) sees = A.mask[(int64_t)s.r * A.T + (s.row0 + wrow) / A.G.g] & low_bits(s.cnt);
    for (int32_t i = 0; i < n; ++i) {
      uint32_t vis[kTile / 32] = {(uint32_t)sees, (uint32_t)(sees >> 32)};  // who the row sees of the tile
      bool gaps = false, masked = true;
      if (i >= lead) {
        const uint16_t tile = tiles[s.part + (i - lead) * split];
        gaps = masked = !(tile & kWhole) || tt < kTile;
        if (gaps) {
          const int32_t slot0 = tile_of(tile) * spt;
#pragma unroll
          for (int u = 0; u < kTile / 32; ++u) {
            const int32_t tok = lane + 32 * u, slot = slot0 + tok / bs;
            vis[u] = __ballot_sync(0xffffffffu, tok < tt && slot < A.G.kb && tok % bs < nv[min(slot, A.G.kb - 1)]);
          }
        }
      }
      if (!warp_wait(B.s_full[w][i & 1], (i >> 1) & 1)) {
        fail(2);
        break;
      }
      // With two S buffers, S of tile i follows O of tile i - 2, so this passes at once; it keeps each barrier's
      // waits in step with its phases, where tile i - 1's below is waited for only now and then
      if (kS == 2 && i > 1 && !warp_wait(B.pv_done[w][i & 1], ((i - 2) >> 1) & 1)) {
        fail(6);
        break;
      }
      tc_fence_after();
      if (gaps || (i < lead && (bad || s.cnt < A.T))) {
        // Lines of the V tile that hold no valid token may hold anything: zero them before the product, and so
        // the drafted values that are not finite. Each warpgroup does, whichever product comes first.
        if (!warp_wait(B.full[v_use(i) % ring], (v_use(i) / ring) & 1)) {
          fail(4);
          break;
        }
        constexpr int kPieces = D / 8;
        uint8_t* v = rs + (size_t)(v_use(i) % ring) * L::kBuf;
        auto vis_of = [&](int u) {
          uint32_t x = vis[0];
#pragma unroll
          for (int k = 1; k < kTile / 32; ++k)
            if (u == k) x = vis[k];
          return x;
        };
        if (i < lead) {
#pragma unroll 1
          for (int e = row; e < A.T * kPieces; e += 128) {
            const int j = e / kPieces;
            if (j < s.cnt && !(bad >> j & 1)) continue;
            uint4* x = reinterpret_cast<uint4*>(v + L::piece(j, e % kPieces));
            uint4 y = make_uint4(0, 0, 0, 0);
            if (j < s.cnt) {
              y = *x;
              clean(y);
            }
            *x = y;
          }
        } else {
#pragma unroll 1
          for (int u = 0; u < kTile / 32; ++u)
            for (int e = row; e < 32 * kPieces; e += 128) {
              const int j = e / kPieces, c = e % kPieces;
              if (!(vis_of(u) >> j & 1)) *reinterpret_cast<uint4*>(v + L::piece(32 * u + j, c)) = make_uint4(0, 0, 0, 0);
            }
        }
        __syncwarp();
        fence_proxy_async();
      }
      bool lost = false;
      if (active) {
        const uint32_t st = my + (kS == 2 ? (i & 1) * kTile : 0);
        uint32_t a[32], b[32];
        // 64 scores of the row from column c on; those it does not see as -infinity
        auto scores = [&](int c) {
          tmem_ld32(a, st + c);
          tmem_ld32(b, st + c + 32);
          tmem_wait_ld(a);
          tmem_wait_ld(b);
          if (masked) {
            const uint32_t lo = vis[c / 32], hi = vis[c / 32 + 1];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(lo >> e & 1)) a[e] = 0xFF800000u;
              if (!(hi >> e & 1)) b[e] = 0xFF800000u;
            }
          }
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = kTile - 64; c >= 0; c -= 64) {  // the first 64 last: they stay in registers for the weights
          scores(c);
#pragma unroll
          for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], fmaxf(__uint_as_float(a[e]), __uint_as_float(b[e])));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        if (__any_sync(0xffffffffu, top > m_run + 8.f)) {
          const float mn = fmaxf(m_run, top);  // of every row of the warp: the next vote is then far off
          const float f = m_run == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : ex2(m_run - mn);
          m_run = mn;
          l_run *= f;
          if (i > 0) {
            // O has the products of tile i - 1; with one S buffer those came before S of this tile
            if (kS == 2) lost = !warp_wait(B.pv_done[w][(i - 1) & 1], ((i - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              uint32_t o[32];
              tmem_ld32(o, my + kO + k);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(my + kO + k, o);
            }
          }
        }
        const float neg = m_run == -INFINITY ? 0.f : -m_run;
        const float2 scale2 = make_float2(scale, scale), neg2 = make_float2(neg, neg);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < kTile; c += 64) {
          if (c > 0) scores(c);
          uint32_t p[32];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 x = fma2(make_float2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])), scale2, neg2);
            float2 y = fma2(make_float2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])), scale2, neg2);
            x = make_float2(ex2(x.x), ex2(x.y));
            y = make_float2(ex2(y.x), ex2(y.y));
            sum0 = add2(sum0, x);
            sum1 = add2(sum1, y);
            p[e] = pack2(x.x, x.y);
            p[16 + e] = pack2(y.x, y.y);
          }
          tmem_st32(st + c / 2, p);  // over scores that have been read
        }
        sum0 = add2(sum0, sum1);
        l_run += sum0.x + sum0.y;
        tmem_wait_st();
      }
      if (lost) {
        fail(3);
        break;
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&B.p_full[w][i & 1]));
    }
    if (n > 0 && !warp_wait(B.pv_done[w][(n - 1) & 1], ((n - 1) >> 1) & 1)) fail(5);
    tc_fence_after();
  }
  __syncthreads();  // every product done: the ring and Q become the cluster's partials
  const bool failed = *(volatile int32_t*)&B.failed != 0;
  if (warp < NW * 4) {
    const int w = warp >> 2, row = tid & 127, wrow = w * gr + row, mrow = s.row0 + wrow;
    const bool real = row < gr && wrow < s.rows;
    const int32_t rows = min(gr, s.rows - w * gr) - (warp & 3) * 32;  // of this warp
    const uint32_t my = tmem + w * kCols + ((uint32_t)(warp & 3) << 21) + kO;
    if (rows > 0 && split == 1 && !failed) {
      // through shared memory (this warp's rows in the place of its queries), to write whole lines
      constexpr int kPieces = D / 8, kXor = kPieces % 8 ? 3 : 7;  // pieces of eight rows on different banks
      uint8_t* mine = qs + ((size_t)w * q_rows + (warp & 3) * 32) * D * 2;
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      const uint64_t bad = B.bad && real ? B.bad & A.mask[(int64_t)s.r * A.T + mrow / A.G.g] : 0;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(o, my + c);
        tmem_wait_ld(o);
        if (!real) continue;
        if (l_run == 0.f) {  // no weights (but infinite values, perhaps)
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float4 x = make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv, __uint_as_float(o[e + 2]) * inv,
                                 __uint_as_float(o[e + 3]) * inv);
          float4 y = make_float4(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv, __uint_as_float(o[e + 6]) * inv,
                                 __uint_as_float(o[e + 7]) * inv);
          if (bad) {
            add_not_finite<__nv_bfloat16>(A, s, bad, c + e, x);
            add_not_finite<__nv_bfloat16>(A, s, bad, c + e + 4, y);
          }
          *reinterpret_cast<uint4*>(mine + ((size_t)lane * kPieces + (((c + e) / 8) ^ (lane & kXor))) * 16) =
              make_uint4(pack2(x.x, x.y), pack2(x.z, x.w), pack2(y.x, y.y), pack2(y.z, y.w));
        }
      }
      __syncwarp();
      const uint32_t per_g = (65536 + A.G.g - 1) / A.G.g;  // m * per_g >> 16 is m / g for the rows there are
      const int32_t m0 = s.row0 + w * gr + (warp & 3) * 32;
      __nv_bfloat16* base = (__nv_bfloat16*)A.out + row_offset(A, s, 0);
#pragma unroll 4
      for (int e = lane; e < min(rows, 32) * kPieces; e += 32) {
        const int r = e / kPieces, c = e - r * kPieces;
        const uint32_t m = m0 + r, t = m * per_g >> 16;
        const uint4 x = *reinterpret_cast<const uint4*>(mine + ((size_t)r * kPieces + (c ^ (r & kXor))) * 16);
        *reinterpret_cast<uint4*>(base + (t * A.G.Hq + (m - t * A.G.g)) * D + c * 8) = x;
      }
    } else if (rows > 0 && split > 1) {
      float* ml = reinterpret_cast<float*>(qs);
      if (real) {
        ml[wrow] = failed ? -INFINITY : m_run;
        ml[NW * q_rows + wrow] = failed ? 0.f : l_run;
      }
      if (n > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(o, my + c);
          tmem_wait_ld(o);
          if (!real) continue;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(rs + part_chunk(wrow, (c + e) / 4, D, 7)) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
    }
  }
  if (split > 1) {
    const Partial P{smem_u32(rs), smem_u32(qs), smem_u32(qs) + (uint32_t)(NW * q_rows * 4), smem_u32(&B.bad)};
    merge_cluster<__nv_bfloat16>(A, s, P, 7);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == NW * 4 + 1) {
    tc_fence_after();
    tmem_free(tmem, kCols * NW);
  }
}

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

cudaLaunchConfig_t cluster_config(int64_t ctas, int threads, size_t smem, int32_t split, cudaStream_t s, cudaLaunchAttribute (&at)[2]) {
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
__global__ void room_kernel() {}

// CTAs of clusters of c that run at once, for c = 2 .. 12, where an SM holds per_sm of them: a property of the device
// (a cluster stays within a GPC), asked for once per thread.
struct ClusterRoom {
  int threads, per_sm, dev;
  int64_t ctas[kMaxSplit + 1];
};
const ClusterRoom& cluster_room(int threads, int32_t per_sm) {
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
  cudaFuncSetAttribute(room_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  cudaFuncSetAttribute(room_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int32_t c = 2; c <= kMaxSplit; ++c) {
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg = cluster_config(c, threads, 233472 / per_sm - 1024, c, nullptr, at);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, room_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    r.ctas[c] = (int64_t)n * c;
  }
  return r;
}

// What a launch costs, in tile times of a CTA alone on its SM: an item takes its tiles, `fixed` more, and `join`
// more where its CTAs merge; beyond `dense` CTAs per SM more of them finish no more tiles in a time. From launches of
// every split: bf16, d 128, 2048 tokens, 16 rows x 4: 0.76 us a tile of 64, and 152 tiles in that time is HBM's rate;
// 512 rows: 2.1 us a tile of 128; binary32, 64 rows: 4.4 us a tile, two CTAs on an SM hide each other's waits. Every head
// size takes these: a shape of the next cost gives the same result, later by what the fixed parts differ.
struct Costs {
  double fixed, join, dense;
};
constexpr Costs kMmaCosts{5.5, 6, 1}, kMmaCostsWide{1, 6, 1}, kF32Costs{2.8, 0.5, 1.3};

double wave_cost(int64_t ctas, double tiles, const Costs& t, int64_t sms) {
  const double crowd = (double)ctas / ((double)sms * t.dense);
  return tiles * (crowd > 1 ? crowd : 1) + t.fixed;
}

// The shape of least cost, of equal ones the one with more CTAs. Items that fill the GPU go whole and the last ones
// split, in pairs: a larger cluster waits behind whole items until all of its CTAs find a place (48 requests of 16
// tokens: 72 us in pairs, 78 whole or in threes; 12 requests: 21 us in threes, 25 in pairs, 29 whole; one of 8 tokens
// 9.2 in twelves, 9.9 in eights, 10.8 in sixteens, which start late; in binary32, one of 4: 19.8, 28.7 and 20.8).
Shape pick_shape(int64_t items, int32_t groups, int32_t per_sm, int32_t tiles, const Costs& t, const ClusterRoom& room) {
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

template <int DV, int RG>
cudaError_t run_f32(const TreeArgs& A, int32_t n_active, cudaStream_t s) {
  const int32_t spt = kTile / A.G.bs, tiles = (A.G.kb + spt - 1) / spt;
  const int32_t groups = (A.T * A.G.g + 16 * RG - 1) / (16 * RG);
  const size_t smem = f32_smem(DV * 32, RG, A.G.kb, tiles);
  int32_t per_sm = (int32_t)(228 * 1024 / (smem + 1024));
  if (per_sm > f32_ctas(DV)) per_sm = f32_ctas(DV);
  if (per_sm < 1) per_sm = 1;
  const int64_t items = (int64_t)n_active * A.G.Hkv * groups;
  const Shape shape = pick_shape(items, groups, per_sm, tiles, kF32Costs, cluster_room(kF32Threads, per_sm));
  return launch_cluster(tree_f32_kernel<DV, RG>, items, shape, kF32Threads, smem, s, A, shape);
}

template <int DV>
cudaError_t run_f32_rows(const TreeArgs& A, int32_t n_active, cudaStream_t s) {
  return A.T * A.G.g <= 16 ? run_f32<DV, 1>(A, n_active, s) : run_f32<DV, 2>(A, n_active, s);
}

cudaError_t run_f32_d(const TreeArgs& A, int32_t n_active, cudaStream_t s) {
  switch (A.G.d / 32) {
    case 1: return run_f32_rows<1>(A, n_active, s);
    case 2: return run_f32_rows<2>(A, n_active, s);
    case 3: return run_f32_rows<3>(A, n_active, s);
    case 4: return run_f32_rows<4>(A, n_active, s);
    case 5: return run_f32_rows<5>(A, n_active, s);
    case 6: return run_f32_rows<6>(A, n_active, s);
    case 7: return run_f32_rows<7>(A, n_active, s);
    default: return run_f32_rows<8>(A, n_active, s);
  }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
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

// Maps of 5 dims over lines and chunks: the pool as [slots][K, V][tokens], a box of one chunk of the tokens of
// a tile's slots; the queries as [tokens][KV heads][group], a box of q_tok tokens of a KV head; drafted keys
// and values as [tokens][KV heads], a box of a request's T tokens of a head.
template <int D, int NW>
cudaError_t make_maps(const TreeArgs& A, int32_t spt, int32_t q_tok, MmaMaps* m) {
  using L = Lines<D, NW>;
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  auto encode = [&](CUtensorMap* map, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[3], const cuuint32_t (&box)[3]) {
    const cuuint64_t d[5] = {(cuuint64_t)L::kElems, (cuuint64_t)L::kChunks, dims[0], dims[1], dims[2]};
    const cuuint64_t st[4] = {(cuuint64_t)L::kBytes, strides[0], strides[1], strides[2]};
    const cuuint32_t b[5] = {(cuuint32_t)L::kElems, 1, box[0], box[1], box[2]}, step[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), d, st, b, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              L::kElems == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t token = (cuuint64_t)D * 2, half = token * A.G.bs, all = (cuuint64_t)A.G.R * A.T;
  const cuuint64_t g = A.G.g, hkv = A.G.Hkv, bs = A.G.bs;
  const bool ok = encode(&m->pool, A.pool, {bs, 2, (cuuint64_t)A.pool_rows}, {token, half, 2 * half}, {(cuuint32_t)bs, 1, (cuuint32_t)spt}) &&
                  encode(&m->q, A.q, {g, hkv, all}, {token, token * g, token * g * hkv}, {(cuuint32_t)g, 1, (cuuint32_t)q_tok}) &&
                  encode(&m->k, A.k, {hkv, all, 1}, {token, token * hkv, token * hkv * all}, {1, (cuuint32_t)A.T, 1}) &&
                  encode(&m->v, A.v, {hkv, all, 1}, {token, token * hkv, token * hkv * all}, {1, (cuuint32_t)A.T, 1});
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int NW>
cudaError_t run_mma(const TreeArgs& A, int32_t n_active, cudaStream_t s) {
  using L = Lines<D, NW>;
  const int32_t spt = L::kTile / A.G.bs, tiles = (A.G.kb + spt - 1) / spt;
  // a warpgroup's rows: all heads of as many drafted tokens as fit 128
  const int32_t q_tok = A.T < 128 / A.G.g ? A.T : 128 / A.G.g, gr = q_tok * A.G.g, q_rows = (gr + 7) / 8 * 8;
  const int32_t groups = (A.T * A.G.g + NW * gr - 1) / (NW * gr);
  // Two CTAs on an SM where TMEM allows (2 x 256 columns), else one: the ring takes what is left of
  // that share of the shared memory. It is never so small that a third CTA, or one of 256 columns beside one of 512, could
  // come to wait for TMEM (two clusters that each hold what the other waits for would wait for ever).
  const bool two = D <= 128 && NW == 1;
  const size_t share = two ? 115712 : kMaxSmem, rest = 1024 + (size_t)NW * q_rows * D * 2 + mma_misc(A.G.kb, tiles);
  int32_t ring = (int32_t)((share - rest) / L::kBuf);
  if (ring > kMaxRing) ring = kMaxRing;
  size_t smem = rest + (size_t)ring * L::kBuf;
  const size_t third = 233472 / 3, least = two ? third : 2 * third;
  if (smem < least) smem = least;
  const int64_t items = (int64_t)n_active * A.G.Hkv * groups;
  const int32_t per_sm = two ? 2 : 1;
  const Shape shape = pick_shape(items, groups, per_sm, tiles, NW == 1 ? kMmaCosts : kMmaCostsWide, cluster_room(NW * 160 + 32, per_sm));
  MmaMaps maps;
  if (cudaError_t e = make_maps<D, NW>(A, spt, q_tok, &maps)) return e;
  return launch_cluster(tree_mma_kernel<D, NW>, items, shape, NW * 160 + 32, smem, s, A, maps, shape, ring, q_tok, q_rows);
}

cudaError_t run_mma_d(const TreeArgs& A, int32_t n_active, cudaStream_t s) {
  const bool wide = A.T * A.G.g > 128;
  switch (A.G.d) {
    case 32: return wide ? run_mma<32, 2>(A, n_active, s) : run_mma<32, 1>(A, n_active, s);
    case 64: return wide ? run_mma<64, 2>(A, n_active, s) : run_mma<64, 1>(A, n_active, s);
    case 96: return wide ? run_mma<96, 2>(A, n_active, s) : run_mma<96, 1>(A, n_active, s);
    case 128: return wide ? run_mma<128, 2>(A, n_active, s) : run_mma<128, 1>(A, n_active, s);
    case 160: return run_mma<160, 1>(A, n_active, s);
    case 192: return run_mma<192, 1>(A, n_active, s);
    case 224: return run_mma<224, 1>(A, n_active, s);
    default: return run_mma<256, 1>(A, n_active, s);
  }
}

}  // namespace

cudaError_t launch_attend_tree(const TreeArgs& A, int32_t n_active, cudaStream_t s) {
  if (n_active <= 0) return cudaSuccess;
  return A.G.dtype == OKV_F32 ? run_f32_d(A, n_active, s) : run_mma_d(A, n_active, s);
}

}  // namespace okv

extern "C" okv_status okv_attend_tree_static(int32_t n_requests, int32_t n_draft, int32_t q_heads, int32_t kv_heads,
                                             int32_t head_dim, int32_t block_size, int32_t slots, int32_t dtype,
                                             const void* pool, const int32_t* slot_block, const int32_t* lengths,
                                             const int32_t* counts, const void* q, const void* k_draft,
                                             const void* v_draft, const uint64_t* mask, void* out, void* stream) {
  using namespace okv;
  Geom G{};
  if (!tree_geom(n_requests, q_heads, kv_heads, head_dim, block_size, slots, dtype, &G)) return OKV_EINVAL;
  if (n_draft <= 0 || n_draft > 64 || (int64_t)n_requests * n_draft > INT32_MAX) return OKV_EINVAL;
  if (!pool || !slot_block || !lengths || !q || !k_draft || !v_draft || !mask || !out) return OKV_EINVAL;
  if (!aligned16(pool) || !aligned16(q) || !aligned16(k_draft) || !aligned16(v_draft) || !aligned16(out)) return OKV_EINVAL;
  if (okv_status st = check_stream(stream)) return st;
  TreeArgs A{};
  A.G = G;
  A.T = n_draft;
  A.pool = (const uint8_t*)pool;
  A.slot_block = slot_block;
  A.len = lengths;
  A.counts = counts;
  A.q = q;
  A.k = k_draft;
  A.v = v_draft;
  A.mask = mask;
  A.out = out;
  A.pool_rows = (int64_t)n_requests * kv_heads * slots;
  return launch_attend_tree(A, n_requests, (cudaStream_t)stream) == cudaSuccess ? OKV_OK : OKV_ECUDA;
}
