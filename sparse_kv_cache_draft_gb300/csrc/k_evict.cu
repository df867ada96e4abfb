// Slots of a paged pool for the blocks of new tokens: empty ones first, then those whose tokens have drawn the least
// attention weight.
//
// A warp takes a unit (request, KV head), its slots' ids and weights in registers, slot 32 u + lane in round u. The m-th smallest
// weight is found bit by bit over the weights' ordered images, from the highest bit in which any two differ (sorting
// them would move every slot), and slots of that weight go by their index. Everything is integer work on a few
// kilobytes: a call is a launch and two rounds of memory.
#include "okv_tree.h"
#include "tc5.cuh"

namespace okv {
namespace {

constexpr int kWarps = 4;      // units of a CTA
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

template <int N>  // rounds: slots up to 32 N
__global__ void __launch_bounds__(kWarps * 32) evict_kernel(const EvictArgs A) {
  __shared__ uint32_t held_of[kWarps][kRange / 32];
  __shared__ uint16_t new_of[kWarps][32 * N];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* held = held_of[warp];
  uint16_t* fresh = new_of[warp];
  for (int i = lane; i < kRange / 32; i += 32) held[i] = 0;
  grid_wait();
  grid_go();
  const int64_t ua = (int64_t)blockIdx.x * kWarps + warp;
  if (ua >= (int64_t)A.R * A.Hkv) return;
  const int32_t r = (int32_t)(ua / A.Hkv), kb = A.kb, bs = A.bs;
  const int64_t at = ua * kb;
  int32_t id[N];
  float w[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int32_t i = 32 * u + lane;
    id[u] = i < kb ? A.slot_block[at + i] : -1;
    w[u] = i < kb ? A.weight[at + i] : 0.f;
  }
  const int32_t len = A.len[r];
  const bool left_out = len < 0 || (int64_t)len + A.T > INT32_MAX;
  const int32_t n = left_out ? 0 : A.counts ? min(max(A.counts[r], 0), A.T) : A.T;
  const int32_t begin = (int32_t)(((int64_t)max(len, 0) + bs - 1) / bs), stop = (int32_t)(((int64_t)max(len, 0) + n + bs - 1) / bs);
  const int32_t base = max(begin, stop - kRange), span = stop - base;

  // which slots may be taken, and which new blocks there are already
  uint32_t empty = 0, old = 0, key[N];  // bit u: the slot of round u
  __syncwarp();
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int32_t b = id[u];
    const int64_t first = (int64_t)b * bs;
    key[u] = image_of(w[u]);
    if (32 * u + lane >= kb) continue;
    if (b < 0 || (first >= len && b >= stop)) {
      empty |= 1u << u;
    } else if (first >= len) {
      if (b >= base) atomicOr(&held[(b - base) >> 5], 1u << ((b - base) & 31));
    } else if (first >= A.sinks && first + bs <= (int64_t)len - A.recent) {
      old |= 1u << u;
    }
  }
  __syncwarp();
  uint32_t want[2];  // of new blocks base + 64 lane ..
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int32_t left = span - (2 * lane + k) * 32;
    want[k] = ~held[2 * lane + k] & (left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u);
  }
  const int32_t mine = __popc(want[0]) + __popc(want[1]);
  int32_t before = mine;
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const int32_t x = __shfl_up_sync(0xffffffffu, before, k);
    if (lane >= k) before += x;
  }
  const int32_t wanted = __shfl_sync(0xffffffffu, before, 31);
  const int32_t n_empty = __reduce_add_sync(0xffffffffu, __popc(empty)), n_old = __reduce_add_sync(0xffffffffu, __popc(old));
  const int32_t m = min(wanted, n_empty + n_old);
  uint32_t taken = 0;
  if (m > 0) {
    // the m newest of them, in order
    int32_t nth = before - mine - (wanted - m);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (uint32_t x = want[k]; x; x &= x - 1, ++nth)
        if (nth >= 0) fresh[nth] = (uint16_t)((2 * lane + k) * 32 + __ffs(x) - 1);
    const uint32_t below = (1u << lane) - 1u;
    // `from` of the slots with their bit in `of`, by index
    auto take = [&](uint32_t of, int32_t from) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const uint32_t all = __ballot_sync(0xffffffffu, of >> u & 1);
        if ((of >> u & 1) && __popc(all & below) < from) taken |= 1u << u;
        from -= __popc(all);
      }
    };
    take(empty, m);
    const int32_t need = m - n_empty;
    if (need > 0) {
      uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (old >> u & 1) lo = min(lo, key[u]), hi = max(hi, key[u]);
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      // the need-th smallest image: the bits that all share, then bit by bit
      const int bits = 32 - __clz(lo ^ hi);
      uint32_t kth = bits == 32 ? 0u : lo >> bits << bits;
      int32_t less = 0;  // slots below kth
      for (int bit = bits - 1; bit >= 0; --bit) {
        const uint32_t up = kth | 1u << bit;
        int32_t c = 0;
#pragma unroll
        for (int u = 0; u < N; ++u) c += (old >> u & 1) && key[u] < up;
        c = __reduce_add_sync(0xffffffffu, c);
        if (c < need) kth = up, less = c;
      }
      uint32_t same = 0;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (!(old >> u & 1)) continue;
        if (key[u] < kth) taken |= 1u << u;
        if (key[u] == kth) same |= 1u << u;
      }
      take(same, need - less);
    }
    __syncwarp();
    int32_t rank = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const uint32_t all = __ballot_sync(0xffffffffu, taken >> u & 1);
      if (taken >> u & 1) {
        id[u] = base + fresh[rank + __popc(all & below)];
        w[u] = 0.f;
      }
      rank += __popc(all);
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int32_t i = 32 * u + lane;
    if (i >= kb) continue;
    A.slot_block_out[at + i] = id[u];
    A.weight_out[at + i] = w[u];
  }
}

template <int N>
cudaError_t run(const EvictArgs& A, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(((int64_t)A.R * A.Hkv + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_attr(s, attr);
  return cudaLaunchKernelEx(&cfg, evict_kernel<N>, A);
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
  const cudaError_t e = slots <= 32 ? run<1>(A, s) : slots <= 128 ? run<4>(A, s) : slots <= 256 ? run<8>(A, s) : slots <= 512 ? run<16>(A, s) : run<32>(A, s);
  return e == cudaSuccess ? OKV_OK : OKV_ECUDA;
}
