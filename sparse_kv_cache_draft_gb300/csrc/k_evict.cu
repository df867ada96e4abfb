// Slots of a paged pool for the blocks of new tokens: empty ones first, then those whose tokens have drawn the least
// attention weight.
//
// A unit (request, KV head) is a warp's up to 128 slots, four to a thread, and a CTA's beyond, one to a thread, ids and
// weights in registers. The m-th smallest weight is found bit by bit over the weights' ordered images, from the highest bit in
// which any two differ (sorting them would move every slot), and slots of that weight go by their index. Everything is
// integer work on a few kilobytes: a call is a launch, two rounds of memory and the sums over the unit. Measured: 128 requests x 8
// heads of 128 slots, a sixteenth of which need one, 2.9 to 4.4 us (by the host's rate of calls); 16 x 8 of 1024 slots for 63 blocks each 8.3 us.
#include "okv_tree.h"
#include "tc5.cuh"

namespace okv {
namespace {

constexpr int kUnits = 4;      // of a CTA, of a warp each
constexpr int kRange = 2048;   // new blocks looked at: the last kb that no slot holds are among the last 2 kb
constexpr int kMaxSlots = 1024;

struct EvictArgs {
  int32_t R, Hkv, bs, kb, T, sinks, recent;
  const int32_t *len, *counts;
  const int32_t* slot_block;
  const float* weight;
  int32_t* slot_block_out;
  float* weight_out;
};

// Ascending as the numbers are, zeros of both signs alike and NaN above all.
__device__ __forceinline__ uint32_t image_of(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

// What a unit's W warps know together.
template <int N, int W>
struct Unit {
  static_assert(W == 1 || N == 1, "a slot to a thread");
  int32_t* x;  // [W]
  int warp;
  __device__ __forceinline__ int32_t count(int32_t mine) { return W == 1 ? __reduce_add_sync(0xffffffffu, mine) : __syncthreads_count(mine); }
  // what the warps before this one have; `all` is a warp's
  __device__ __forceinline__ int32_t before(int32_t all) {
    if (W == 1) return 0;
    const int lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) x[warp] = all;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warp ? x[lane] : 0);
  }
};

// The need-th smallest of the images of a warp's slots, K to a lane (0xFFFFFFFF: none), and how many are below it: the bits that
// all share, then bit by bit.
struct Kth {
  uint32_t image;
  int32_t less;
};
template <int K>
__device__ __forceinline__ Kth kth_of(const uint32_t (&key)[K], int32_t need) {
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int u = 0; u < K; ++u) lo = min(lo, key[u]), hi = max(hi, key[u]);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  const int bits = 32 - __clz(lo ^ hi);
  Kth k{bits == 32 ? 0u : lo >> bits << bits, 0};
  for (int bit = bits - 1; bit >= 0; --bit) {
    const uint32_t up = k.image | 1u << bit;
    int32_t c = 0;
#pragma unroll
    for (int u = 0; u < K; ++u) c += key[u] < up;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c <= need) k.image = up, k.less = c;
    if (c == need) break;  // the need smallest are those below `up`
  }
  return k;
}

template <int N, int W>  // slots up to 32 N W
__global__ void __launch_bounds__((W == 1 ? kUnits : W) * 32) evict_kernel(const EvictArgs A) {
  constexpr int kHere = W == 1 ? kUnits : 1;
  __shared__ uint32_t held_of[kHere][kRange / 32];
  __shared__ uint16_t new_of[kHere][32 * N * W];
  __shared__ int16_t rank_of[kHere][kRange / 32];
  __shared__ int32_t sums[W], kept_less;
  __shared__ uint32_t keys[W == 1 ? 1 : 32 * W];
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5, here = W == 1 ? threadIdx.x >> 5 : 0;
  const int first_slot = warp * N * 32 + lane;  // and of the new blocks, of which W == 1 takes 32 at a time
  uint32_t* held = held_of[here];
  uint16_t* fresh = new_of[here];
  for (int i = threadIdx.x % (W * 32); i < kRange / 32; i += W * 32) held[i] = 0;
  grid_wait();
  grid_go();
  const int64_t ua = (int64_t)blockIdx.x * kHere + here;
  if (ua >= (int64_t)A.R * A.Hkv) return;  // a warp that has its unit to itself
  const int32_t r = (int32_t)(ua / A.Hkv), kb = A.kb, bs = A.bs;
  const int64_t at = ua * kb;
  int32_t id[N];
  float w[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int32_t i = 32 * u + first_slot;
    id[u] = i < kb ? A.slot_block[at + i] : -1;
    w[u] = i < kb ? A.weight[at + i] : 0.f;
  }
  const int32_t len = A.len[r];
  const bool left_out = len < 0 || (int64_t)len + A.T > INT32_MAX;
  const int32_t n = left_out ? 0 : A.counts ? min(max(A.counts[r], 0), A.T) : A.T;
  const int32_t begin = (int32_t)(((int64_t)max(len, 0) + bs - 1) / bs), stop = (int32_t)(((int64_t)max(len, 0) + n + bs - 1) / bs);
  const int32_t base = max(begin, stop - kRange), span = stop - base;
  auto sync = [] {
    if (W == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  Unit<N, W> unit{sums, warp};

  // which slots may be taken, and which new blocks there are already
  uint32_t empty = 0, old = 0, key[N];  // bit u: the slot of round u
  sync();
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int32_t b = id[u];
    const int64_t first = (int64_t)b * bs;
    key[u] = image_of(w[u]);
    if (32 * u + first_slot >= kb) continue;
    if (b < 0 || (first >= len && b >= stop)) {
      empty |= 1u << u;
    } else if (first >= len) {
      if (b >= base) atomicOr(&held[(b - base) >> 5], 1u << ((b - base) & 31));
    } else if (first >= A.sinks && first + bs <= (int64_t)len - A.recent) {
      old |= 1u << u;
    }
  }
  sync();
  uint32_t want[2];  // of new blocks base + 64 lane .., by every warp
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int32_t left = span - (2 * lane + k) * 32;
    want[k] = ~held[2 * lane + k] & (left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u);
  }
  const int32_t mine = __popc(want[0]) + __popc(want[1]);
  const int32_t wanted = __reduce_add_sync(0xffffffffu, mine);
  uint32_t taken = 0;
  if (wanted > 0) {  // the unit's as a whole
    const int32_t n_empty = unit.count(__popc(empty)), n_old = unit.count(__popc(old)), m = min(wanted, n_empty + n_old);
    // the m newest of them, in order: each bit's rank from those of the words before it
    int32_t up = mine;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int32_t x = __shfl_up_sync(0xffffffffu, up, k);
      if (lane >= k) up += x;
    }
    sync();  // `held` has been read
    if (warp == 0) {
      held[2 * lane] = want[0], held[2 * lane + 1] = want[1];
      rank_of[here][2 * lane] = (int16_t)(up - mine), rank_of[here][2 * lane + 1] = (int16_t)(up - __popc(want[1]));
    }
    sync();
    for (int32_t i = first_slot; i < span; i += 32 * W) {
      const uint32_t word = held[i >> 5];
      const int32_t nth = rank_of[here][i >> 5] + __popc(word & ((1u << (i & 31)) - 1u)) - (wanted - m);
      if ((word >> (i & 31) & 1) && nth >= 0) fresh[nth] = (uint16_t)i;
    }
    const uint32_t below = (1u << lane) - 1u;
    // each slot with its bit in `of`, by index: use(u, how many there are before it)
    auto each = [&](uint32_t of, auto use) {
      int32_t rank = unit.before(__reduce_add_sync(0xffffffffu, __popc(of)));
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const uint32_t all = __ballot_sync(0xffffffffu, of >> u & 1);
        if (of >> u & 1) use(u, rank + __popc(all & below));
        rank += __popc(all);
      }
    };
    each(empty, [&](int u, int32_t rank) { taken |= (uint32_t)(rank < m) << u; });
    const int32_t need = m - n_empty;
    if (need > 0) {
      Kth k;
      if constexpr (W == 1) {
#pragma unroll
        for (int u = 0; u < N; ++u)
          if (!(old >> u & 1)) key[u] = 0xFFFFFFFFu;
        k = kth_of(key, need);
      } else {
        // by one warp: an exchange of all for each bit takes longer than a warp's look at all slots (1024 of them 10 us)
        keys[threadIdx.x] = old ? key[0] : 0xFFFFFFFFu;
        __syncthreads();
        if (warp == 0) {
          uint32_t all[W];
#pragma unroll
          for (int u = 0; u < W; ++u) all[u] = keys[32 * u + lane];
          k = kth_of(all, need);
          if (lane == 0) sums[0] = (int32_t)k.image, kept_less = k.less;
        }
        __syncthreads();
        k = Kth{(uint32_t)sums[0], kept_less};
      }
      uint32_t same = 0;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (!(old >> u & 1)) continue;
        if (key[u] < k.image) taken |= 1u << u;
        if (key[u] == k.image) same |= 1u << u;
      }
      each(same, [&](int u, int32_t rank) { taken |= (uint32_t)(rank < need - k.less) << u; });
    }
    sync();
    each(taken, [&](int u, int32_t rank) {
      id[u] = base + fresh[rank];
      w[u] = 0.f;
    });
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int32_t i = 32 * u + first_slot;
    if (i >= kb) continue;
    A.slot_block_out[at + i] = id[u];
    A.weight_out[at + i] = w[u];
  }
}

template <int N, int W>
cudaError_t run(const EvictArgs& A, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg{};
  const int64_t units = (int64_t)A.R * A.Hkv;
  cfg.gridDim = dim3((unsigned)(W == 1 ? (units + kUnits - 1) / kUnits : units));
  cfg.blockDim = dim3((W == 1 ? kUnits : W) * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_attr(s, attr);
  return cudaLaunchKernelEx(&cfg, evict_kernel<N, W>, A);
}

}  // namespace
}  // namespace okv

extern "C" okv_status okv_evict_static(int32_t n_requests, int32_t n_new, int32_t kv_heads, int32_t block_size, int32_t slots,
                                       const int32_t* lengths, const int32_t* counts, int32_t sinks, int32_t recent,
                                       const int32_t* slot_block, const float* weight, int32_t* slot_block_out, float* weight_out,
                                       void* stream) {
  using namespace okv;
  if (n_requests <= 0 || n_new <= 0 || kv_heads <= 0 || block_size <= 0 || block_size > 64 || slots <= 0 || slots > kMaxSlots) return OKV_EINVAL;
  if ((int64_t)n_requests * kv_heads * slots > INT32_MAX || sinks < 0 || recent < 0) return OKV_EINVAL;
  if (!lengths || !slot_block || !weight || !slot_block_out || !weight_out) return OKV_EINVAL;
  if (okv_status st = check_stream(stream)) return st;
  const EvictArgs A{n_requests, kv_heads, block_size, slots, n_new, sinks, recent, lengths, counts, slot_block, weight, slot_block_out, weight_out};
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = slots <= 32 ? run<1, 1>(A, s) : slots <= 128 ? run<4, 1>(A, s) : slots <= 256 ? run<1, 8>(A, s) : slots <= 512 ? run<1, 16>(A, s) : run<1, 32>(A, s);
  return e == cudaSuccess ? OKV_OK : OKV_ECUDA;
}
