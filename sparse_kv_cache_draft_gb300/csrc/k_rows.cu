// Rows of a projection on their way to the attention and the cache: per-head RMS norm of queries and
// keys, position rotation, and the append of keys and values to the paged store.
//
// A row holds Hq query heads, Hkv key heads and Hkv value heads of d elements. For a query or key
// head x at position p, with weight w (the norm is left out without one):
//   y = x / sqrt(mean(x^2) + eps) * w
//   (y_a, y_b) <- (y_a cos t_i - y_b sin t_i, y_b cos t_i + y_a sin t_i),  t_i = p inv_freq_i
// for the rotated pairs i, (a, b) = (i, i + half) or (2i, 2i + 1); the dims behind the rotated ones
// and the value heads pass. Everything is binary32 with one rounding at the store.
//
// Angles: p inv_freq is reduced to less than a turn before anything is rounded to binary32.
// inv_freq / 2 pi as a 64-bit fraction of a turn, times the integer p modulo 2^64, is the phase, off by
// p 2^-63 turns at most (2^-32 turns at position 2^31).
//
// The rows move once in and once out, so HBM is the limit: 16384 rows of 64 / 8 heads of 128 dims in bf16 take
// 111 us, 6.0 TB/s (0.89 of a copy's rate), ragged chunks of 1024 tokens of 16 requests are appended at 0.84. A
// head row is 8 elements on each of d / 8 lanes (a subgroup of the next power of two of lanes). A warp takes a row, or a part of its
// heads where rows are few: it computes the row's angles once, folds weights, cosines and sines into two
// factors per element that stay in registers for all of its query (then key) heads, and keeps 64 bytes a lane
// in flight. What that took, on those 16384 rows: a CTA to a token with its angles in shared memory and a
// division per head row 291 us; a warp to a row and the factors in registers 148; 64 registers, so that 32
// warps share an SM (not 16), and the first loads before the angles 117; loops of their own for queries, keys
// and values, and for the two orders of pairs, 113; a launch that starts while the last one ends 111. Slower: loading each next head row beside the work on the
// last (160 us and more: the loads' scoreboards are shared), and batches of 6 or of 2 (130 to 145).
#include <cuda_bf16.h>

#include "okv_tree.h"
#include "tc5.cuh"

namespace okv {
namespace {

constexpr int kThreads = 256;
template <typename T>
constexpr int kInFlight = 16 / (int)sizeof(T) / 2;  // head rows of each subgroup in flight: 64 bytes a lane

// 8 elements of a head row.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The fraction of a turn that one position adds, in units of 2^-64: f / 2 pi modulo 1, from the 24 bits of
// f's mantissa times 2^66 / 2 pi, shifted to f's exponent. Off by less than 2^-64 and 2^-64 of itself.
__device__ __forceinline__ uint64_t turn_per_position(float f) {
  const uint32_t bits = __float_as_uint(f), ex = bits >> 23 & 255;
  const uint64_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u), k = 11743562013128004906ull;  // round(2^66 / 2 pi)
  const uint64_t hi = __umul64hi(m, k), lo = m * k;
  const int sh = 2 - ((int)(ex ? ex : 1) - 150);  // f = m 2^(ex - 150)
  uint64_t t;
  if (sh >= 128)
    t = 0;
  else if (sh >= 64)
    t = hi >> (sh - 64);
  else if (sh > 0)
    t = hi << (64 - sh) | lo >> sh;
  else
    t = sh > -64 ? lo << -sh : 0;
  return bits >> 31 ? 0 - t : t;
}
// cos and sin of pos * f radians, `per` being f's turn_per_position.
__device__ __forceinline__ void angle(uint64_t per, float f, int32_t pos, float* c, float* s) {
  const uint64_t phase = per * (uint64_t)(int64_t)pos;
  // the nearest quarter turn, and the rest in half turns, within +-1/4
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const float rest = (float)(int64_t)(phase - ((uint64_t)quarter << 62)) * 1.0842021724855044e-19f;  // 2^-63
  float sv, cv;
  sincospif(rest, &sv, &cv);
  const float a = (quarter & 1) ? sv : cv, b = (quarter & 1) ? cv : sv;
  *c = (quarter == 1 || quarter == 2) ? -a : a;
  *s = quarter >= 2 ? -b : b;
  if (!isfinite(f)) *c = *s = __int_as_float(0x7FC00000);
}

// The turn of one kind of head (queries or keys) at one position, for the 8 dims of a lane: element e of a
// head row x becomes r (x_e wc_e + x'_e ws_e), x' being the other element of its pair, r the norm's root,
// wc the weight times the cosine and ws the other element's weight times the signed sine.
struct Turn {
  float2 wc[4], ws[4];
  int other;       // the lane that holds the pairs' other elements
  bool pair, norm; // this lane's dims are rotated; there is a norm
  float per_d;     // 1 / d
};

// Every lane calls it; `cs`, `sn`: the token's tables of `half` entries.
template <typename T>
__device__ __forceinline__ Turn make_turn(const RowArgs& A, const T* w, const float* cs, const float* sn, int sub) {
  Turn t;
  const int lane = threadIdx.x & 31, step = A.half / 8;  // lanes between the two halves
  const bool low = sub < step;
  t.pair = sub < 2 * step;
  t.norm = w != nullptr;
  t.per_d = 1.f / (float)A.d;
  t.other = A.interleaved || !t.pair ? lane : low ? lane + step : lane - step;
  float c[8], s[8], a[8], b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = a[e] = b[e] = 1.f, s[e] = 0.f;
  if (t.pair) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = A.interleaved ? sub * 4 + e / 2 : (low ? sub : sub - step) * 8 + e;
      c[e] = cs[i];
      s[e] = (A.interleaved ? (e & 1) == 0 : low) ? -sn[i] : sn[i];
    }
  }
  if (w && sub * 8 < A.d) {
    Eight<T> v;
    v.load(w + sub * 8);
    v.get(a);
    v.load(w + (sub + t.other - lane) * 8);
    v.get(b);
    if (A.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = a[e ^ 1];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.wc[e] = make_float2(a[2 * e] * c[2 * e], a[2 * e + 1] * c[2 * e + 1]);
    // dims that are not rotated pass: +0 times -0 adds nothing to them, also not the sign of a zero
    t.ws[e] = t.pair ? make_float2(b[2 * e] * s[2 * e], b[2 * e + 1] * s[2 * e + 1]) : make_float2(-0.f, -0.f);
  }
  return t;
}

// x' of a lane: from the lane that holds it, or the neighbour within the lane. `some`: there are dims that
// are not rotated, whose x' is zero (it may be infinite, and its factor is zero).
template <bool INTER>
__device__ __forceinline__ void others(Eight<__nv_bfloat16>& x, const Turn& t, bool some) {
  uint32_t w[4] = {x.u.x, x.u.y, x.u.z, x.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = INTER ? __byte_perm(w[i], 0, 0x1032) : __shfl_sync(0xffffffffu, w[i], t.other);
  if (some && !t.pair) w[0] = w[1] = w[2] = w[3] = 0;
  x.u = make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool INTER>
__device__ __forceinline__ void others(Eight<float>& x, const Turn& t, bool some) {
  float v[8];
  x.get(v);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = v[i], b = v[i + 1];
    v[i] = INTER ? b : __shfl_sync(0xffffffffu, a, t.other);
    v[i + 1] = INTER ? a : __shfl_sync(0xffffffffu, b, t.other);
  }
  if (some && !t.pair) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  x.set(v);
}

// Norm and rotation of a head row held by the LPG lanes of a subgroup (zeros in lanes past d). Every lane of
// the warp calls it.
template <int LPG, bool INTER, typename T>
__device__ __forceinline__ void norm_turn(const RowArgs& A, Eight<T>& raw, const Turn& t) {
  Eight<T> mate = raw;
  others<INTER>(mate, t, 2 * A.half != A.d);
  float x[8], y[8];
  raw.get(x);
  mate.get(y);
  float2 r = make_float2(1.f, 1.f);
  if (t.norm) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) s2 = fma2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(x[2 * e], x[2 * e + 1]), s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int off = LPG / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    r.x = r.y = rsqrtf(fmaf(ss, t.per_d, A.eps));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 v = mul2(make_float2(x[2 * e], x[2 * e + 1]), t.wc[e]);
    v = mul2(fma2(make_float2(y[2 * e], y[2 * e + 1]), t.ws[e], v), r);
    x[2 * e] = v.x;
    x[2 * e + 1] = v.y;
  }
  raw.set(x);
}

// Where the rows of one launch come from and go to.
struct RowsTo {
  int32_t n_rows;              // norm_rope: rows; append: requests
  int32_t parts;               // warps of a row
  const int32_t* positions;    // norm_rope
  void *k, *v;                 // norm_rope: [rows][Hkv][d] or NULL
  // append
  int32_t n_new, ctas, span;   // ctas of a request; blocks a CTA's tokens may touch
  int32_t bs, kb;
  const int32_t *counts, *len, *slot_block;
  void* pool;                  // [R][Hkv][kb][2][bs][d]
};

template <typename T, int LPG, bool APPEND, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const RowArgs A, const RowsTo R) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32, kSub = 32 / LPG;  // head rows of a warp
  constexpr int kFly = kInFlight<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPG, sg = lane / LPG;
  float* cs = reinterpret_cast<float*>(smem) + warp * 2 * A.half;       // [warps][cos, sin][half]
  float* sn = cs + A.half;
  int32_t* slot_of = reinterpret_cast<int32_t*>(smem) + kWarps * 2 * A.half;  // append: [Hkv][span]
  const bool on = sub * 8 < A.d;
  grid_wait();
  grid_go();

  int64_t row;
  int32_t pos = 0, part, r = 0, blk0 = 0, last = 0;
  bool mine;  // a row of this warp's own (its position may still leave it out)
  constexpr int kAhead = 4;
  int32_t slots[kAhead];  // the first slots of the request's table that this thread looks at
  const int32_t* sb = nullptr;
  if (APPEND) {
    r = blockIdx.x / R.ctas;
    const int32_t w0 = (blockIdx.x - r * R.ctas) * kWarps, t0 = w0 / R.parts, t = (w0 + warp) / R.parts;
    part = (w0 + warp) % R.parts;
    sb = R.slot_block + (int64_t)r * A.Hkv * R.kb;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int32_t i = threadIdx.x + u * kThreads;
      slots[u] = i < A.Hkv * R.kb ? sb[i] : -1;
    }
    const int32_t cnt = R.counts ? min(max(R.counts[r], 0), R.n_new) : R.n_new, len = R.len[r];
    if (t0 >= cnt || len < 0 || len > INT32_MAX - R.n_new) return;  // positions stay within 31 bits
    mine = t < cnt;
    row = (int64_t)r * R.n_new + t;
    pos = len + t;
    blk0 = (len + t0) / R.bs;
    last = (len + min(cnt - 1, (w0 + kWarps - 1) / R.parts)) / R.bs;
  } else {
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    row = w / R.parts;
    part = (int32_t)(w - row * R.parts);
    mine = row < R.n_rows;
    if (mine) pos = R.positions[row];
  }
  // The row's head rows in groups of a warp: queries, keys, values. A warp takes every `parts`-th group, a
  // batch of loads ahead of the work on them; the first ones go out before the slots and the angles.
  const int32_t gq = (A.Hq + kSub - 1) / kSub, gk = (A.Hkv + kSub - 1) / kSub;
  const T* from = (const T*)A.qkv + row * A.row_stride + sub * 8;
  auto load = [&](Eight<T>(&raw)[kFly], int32_t g, int32_t first, int32_t heads, const T* in) {
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int32_t h = (g + u * R.parts - first) * kSub + sg;
      raw[u].zero();
      if (h < heads && on) raw[u].load(in + h * A.d);
    }
  };
  int32_t g = part;
  Eight<T> raw[kFly];
  bool ahead = mine && g < gq && A.q;
  if (ahead) load(raw, g, 0, A.Hq, from);
  if (APPEND) {
    for (int32_t i = threadIdx.x; i < A.Hkv * R.span; i += kThreads) slot_of[i] = INT32_MAX;
    __syncthreads();
    auto match = [&](int32_t i, int32_t b) {
      if (b >= blk0 && b <= last) atomicMin(&slot_of[i / R.kb * R.span + (b - blk0)], i % R.kb);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) match(threadIdx.x + u * kThreads, slots[u]);
    for (int32_t i = threadIdx.x + kAhead * kThreads; i < A.Hkv * R.kb; i += kThreads) match(i, sb[i]);
    __syncthreads();
  }
  if (!mine || pos < 0) return;
  for (int32_t f = lane; f < A.half; f += 32) {
    const float inv = A.inv_freq[f];
    angle(turn_per_position(inv), inv, pos, &cs[f], &sn[f]);
  }
  __syncwarp();
#pragma unroll
  for (int kind = 0; kind < 3; ++kind) {
    const int32_t heads = kind == 0 ? A.Hq : A.Hkv, first = kind == 0 ? 0 : kind == 1 ? gq : gq + gk, end = kind == 0 ? gq : first + gk;
    if (g >= end) continue;
    const T* in = from + (int64_t)(kind == 0 ? 0 : kind == 1 ? A.Hq : A.Hq + A.Hkv) * A.d;
    T* out = nullptr;
    if (kind == 0) {
      if (A.q) out = (T*)A.q + row * A.Hq * A.d + sub * 8;
    } else if (APPEND) {
      out = (T*)R.pool + ((int64_t)r * A.Hkv * R.kb * 2 + kind - 1) * R.bs * A.d + (int64_t)(pos % R.bs) * A.d + sub * 8;
    } else {
      T* to = (T*)(kind == 1 ? R.k : R.v);
      if (to) out = to + row * A.Hkv * A.d + sub * 8;
    }
    if (!out) {
      g += (end - g + R.parts - 1) / R.parts * R.parts;
      continue;
    }
    Turn t;
    if (kind < 2) t = make_turn<T>(A, (const T*)(kind == 0 ? A.q_weight : A.k_weight), cs, sn, sub);
    const int32_t* slot_at = APPEND ? slot_of + (pos / R.bs - blk0) : nullptr;
    const int32_t slot_size = APPEND ? 2 * R.bs * A.d : 0;  // elements
    auto work = [&](Eight<T>(&raw)[kFly], int32_t g) {
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (g + u * R.parts >= end) break;
        if (kind < 2) norm_turn<LPG, INTER, T>(A, raw[u], t);
        const int32_t h = (g + u * R.parts - first) * kSub + sg;
        if (h >= heads || !on) continue;
        int64_t at = h * A.d;  // elements of a row: at most 4096 * 256
        if (APPEND && kind > 0) {
          const int32_t slot = slot_at[h * R.span];
          if (slot == INT32_MAX) continue;
          at = (int64_t)(h * R.kb + slot) * slot_size;
        }
        raw[u].store(out + at);
      }
    };
    for (; g < end; g += kFly * R.parts) {
      if (!ahead) load(raw, g, first, heads, in);
      ahead = false;
      work(raw, g);
    }
    // the last batch may have stepped past groups of the next kind
    while (g - R.parts >= end) g -= R.parts;
  }
}

template <typename T, bool APPEND>
cudaError_t run_rows(const RowArgs& A, RowsTo R, cudaStream_t s) {
  const int d8 = A.d / 8, lpg = d8 <= 4 ? 4 : d8 <= 8 ? 8 : d8 <= 16 ? 16 : 32, heads = 32 / lpg, warps = kThreads / 32;
  const int32_t groups = (A.Hq + heads - 1) / heads + 2 * ((A.Hkv + heads - 1) / heads);
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // Warps of a row: one where there are rows enough for 16 warps on every SM, else as many as reach that, in powers
  // of two, so that a CTA has whole rows or a row whole CTAs, which share a slot table (an append of 128 rows of 32 / 8
  // heads takes 5.4 us with 16, 6.9 with 20; 512 rows 5.9 with 4, 7.9 with 5; 1024 rows 7.5 with 2, 9.5 with 3).
  const int64_t rows = APPEND ? (int64_t)R.n_rows * R.n_new : R.n_rows;
  int64_t parts = ((int64_t)sms * 16 + rows - 1) / rows;
  if (parts >= groups)
    parts = groups;  // a group of heads to a warp (one row: 3.4 us with 24, 4.0 with 16)
  else
    while (parts & (parts - 1)) parts &= parts - 1;
  R.parts = (int32_t)parts;
  int64_t ctas;
  if (APPEND) {
    const int64_t per = ((int64_t)R.n_new * R.parts + warps - 1) / warps;
    ctas = per * R.n_rows;
    R.ctas = (int32_t)per;
    R.span = (warps + R.parts - 1) / R.parts + 1;  // blocks of a CTA's tokens, one token a block at worst
  } else {
    ctas = ((int64_t)R.n_rows * R.parts + warps - 1) / warps;
  }
  const size_t smem = (size_t)warps * A.half * 8 + (APPEND ? (size_t)A.Hkv * R.span * 4 : 0);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    if (smem > 48 * 1024) {
      if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448)) return e;
    }
    cudaLaunchAttribute at;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = overlap_attr(s, &at);
    return cudaLaunchKernelEx(&cfg, kernel, A, R);
  };
  if (A.interleaved)
    return lpg == 4    ? go(rows_kernel<T, 4, APPEND, true>)
           : lpg == 8  ? go(rows_kernel<T, 8, APPEND, true>)
           : lpg == 16 ? go(rows_kernel<T, 16, APPEND, true>)
                       : go(rows_kernel<T, 32, APPEND, true>);
  return lpg == 4    ? go(rows_kernel<T, 4, APPEND, false>)
         : lpg == 8  ? go(rows_kernel<T, 8, APPEND, false>)
         : lpg == 16 ? go(rows_kernel<T, 16, APPEND, false>)
                     : go(rows_kernel<T, 32, APPEND, false>);
}

// ---- a context's append ----------------------------------------------------------------------------

// The token's place in one unit: the host block, the resident slot and the kept copy that hold its
// block (NULL where there is none) and the block's summary.
template <typename T>
struct Places {
  T *host, *pool, *kept, *summ;
  int32_t t;  // token within the block
};

// False (recorded) if the position is past the request's host capacity.
__device__ __forceinline__ bool position_ok(const Geom& G, int32_t layer, int32_t r, int32_t pos, int32_t cap, int32_t* err) {
  if (pos >= 0 && pos < cap * G.bs && pos < G.nb_max * G.bs) return true;
  record_error(err, kErrCapacity, layer, r, pos);
  return false;
}
template <typename T>
__device__ __forceinline__ Places<T> places(const Geom& G, const LayerState& S, const ReqTables& RT, int32_t layer, int32_t r, int32_t h,
                                            int32_t pos, int32_t slot, int32_t* err) {
  const int64_t unit = (int64_t)r * G.Hkv + h;
  const int32_t b = pos / G.bs, lcap = RT.local_cap[r];
  Places<T> p;
  p.t = pos - b * G.bs;
  p.host = reinterpret_cast<T*>(RT.host_kv[r] + (((int64_t)layer * G.Hkv + h) * RT.cap_blocks[r] + b) * G.block_bytes);
  p.pool = slot != INT32_MAX ? reinterpret_cast<T*>(S.pool + (unit * G.kb + slot) * G.block_bytes) : nullptr;
  p.kept = nullptr;
  if (lcap > 0) {
    const int32_t e = S.local_of[unit * G.nb_max + b];
    if (e >= lcap)
      record_error(err, kErrLocalRange, layer, r, e);
    else if (e >= 0)
      p.kept = reinterpret_cast<T*>(RT.local_kv[r] + (((int64_t)layer * G.Hkv + h) * lcap + e) * G.block_bytes);
  }
  p.summ = reinterpret_cast<T*>(S.summ) + (unit * G.nb_max + b) * 2 * G.d;
  return p;
}

// Eight dims of a key (which = 0) or value (1) into every place; a key also into the summary, with
// the comparisons of okv_append (strict, so ties keep the earlier token).
template <typename T>
__device__ __forceinline__ void put(const Geom& G, const Places<T>& p, int which, int32_t c, const Eight<T>& x) {
  const int64_t at = (int64_t)(which * G.bs + p.t) * G.d + c;
  x.store(p.host + at);
  if (p.pool) x.store(p.pool + at);
  if (p.kept) x.store(p.kept + at);
  if (which) return;
  Eight<T> lo = x, hi = x;
  if (p.t > 0) {
    float v[8], a[8], b[8];
    lo.load(p.summ + c);
    hi.load(p.summ + G.d + c);
    x.get(v);
    lo.get(a);
    hi.get(b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (v[e] < a[e]) a[e] = v[e];
      if (v[e] > b[e]) b[e] = v[e];
    }
    lo.set(a);
    hi.set(b);
  }
  lo.store(p.summ + c);
  hi.store(p.summ + G.d + c);
}

// One CTA per active request. Dynamic shared memory: cos and sin [half], slot_of [Hkv].
template <typename T, int LPG>
__global__ void __launch_bounds__(kThreads) append_qkv_kernel(const RowArgs A, const Geom G, const LayerState S, const ReqTables RT,
                                                              const int32_t layer, int32_t* err) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* cs = reinterpret_cast<float*>(smem);
  float* sn = cs + A.half;
  int32_t* slot_of = reinterpret_cast<int32_t*>(sn + A.half);
  const int tid = threadIdx.x, sub = tid % LPG, group = tid / LPG;
  constexpr int kGroups = kThreads / LPG;
  const int32_t r = RT.active[blockIdx.x], pos = S.len[r];
  if (!position_ok(G, layer, r, pos, RT.cap_blocks[r], err)) return;
  for (int32_t i = tid; i < A.Hkv; i += kThreads) slot_of[i] = INT32_MAX;
  __syncthreads();
  const int32_t* sb = S.slot_block + (int64_t)r * G.Hkv * G.kb;
  for (int32_t i = tid; i < G.Hkv * G.kb; i += kThreads)
    if (sb[i] == pos / G.bs) atomicMin(&slot_of[i / G.kb], i % G.kb);
  for (int32_t f = tid; f < A.half; f += kThreads) {
    const float inv = A.inv_freq[f];
    angle(turn_per_position(inv), inv, pos, &cs[f], &sn[f]);
  }
  __syncthreads();
  const T* from = (const T*)A.qkv + (int64_t)r * A.row_stride;
  const bool on = sub * 8 < A.d;
  for (int kind = 0; kind < 3; ++kind) {
    const int32_t heads = kind == 0 ? A.Hq : A.Hkv;
    const T* in = from + (int64_t)(kind == 0 ? 0 : kind == 1 ? A.Hq : A.Hq + A.Hkv) * A.d;
    Turn t;
    if (kind < 2) t = make_turn<T>(A, (const T*)(kind == 0 ? A.q_weight : A.k_weight), cs, sn, sub);
    for (int32_t base = 0; base < heads; base += kGroups) {
      const int32_t h = base + group;
      Eight<T> raw;
      raw.zero();
      if (h < heads && on) raw.load(in + (int64_t)h * A.d + sub * 8);
      if (kind < 2) {
        if (A.interleaved)
          norm_turn<LPG, true, T>(A, raw, t);
        else
          norm_turn<LPG, false, T>(A, raw, t);
      }
      if (h >= heads || !on) continue;
      if (kind == 0)
        raw.store((T*)A.q + ((int64_t)r * A.Hq + h) * A.d + sub * 8);
      else
        put(G, places<T>(G, S, RT, layer, r, h, pos, slot_of[h], err), kind - 1, sub * 8, raw);
    }
  }
  __syncthreads();
  if (tid == 0) {
    S.len[r] = pos + 1;
    S.len_act[blockIdx.x] = pos + 1;
  }
}

// grid (n active requests from P.first on, Hkv), d / 8 lanes at work (the tokens of a block go through its summary in order).
// The last of a request's Hkv CTAs to finish (counted in arrivals[r], zero before and after)
// advances its length.
template <typename T>
__global__ void __launch_bounds__(128) append_tree_kernel(const Geom G, const LayerState S, const ReqTables RT, const int32_t layer, const int32_t n_draft,
                                                          const T* __restrict__ k, const T* __restrict__ v, const __grid_constant__ Accepted P,
                                                          int32_t* __restrict__ arrivals, int32_t* err) {
  const int32_t a = P.first + blockIdx.x, r = RT.active[a], h = blockIdx.y, tid = threadIdx.x;
  const uint8_t* path = P.path + blockIdx.x * P.stride + 1;
  const int32_t n = path[-1];
  if (n <= 0) return;
  const int32_t pos0 = S.len[r];
  __shared__ int32_t slot;
  const int32_t* sb = S.slot_block + ((int64_t)r * G.Hkv + h) * G.kb;
  // the first half of the CTA copies the keys, the second the values
  const int which = tid >> 6, c = (tid & 63) * 8;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t pos = pos0 + i;
    if (!position_ok(G, layer, r, pos, RT.cap_blocks[r], err)) break;  // the same for every thread
    if (i == 0 || pos % G.bs == 0) {
      __syncthreads();
      if (tid == 0) slot = INT32_MAX;
      __syncthreads();
      for (int32_t j = tid; j < G.kb; j += blockDim.x)
        if (sb[j] == pos / G.bs) atomicMin(&slot, j);
      __syncthreads();
    }
    if (c < G.d) {
      const int64_t at = (((int64_t)r * n_draft + path[i]) * G.Hkv + h) * G.d + c;
      Eight<T> x;
      x.load((which ? v : k) + at);
      put(G, places<T>(G, S, RT, layer, r, h, pos, slot, err), which, c, x);
    }
  }
  __threadfence();
  __syncthreads();
  if (tid == 0 && atomicAdd(&arrivals[r], 1) == G.Hkv - 1) {
    arrivals[r] = 0;
    __threadfence();
    S.len[r] = pos0 + n;
    S.len_act[a] = pos0 + n;
  }
}

template <typename T>
cudaError_t run_append_qkv(const RowArgs& A, const Geom& G, const LayerState& S, const ReqTables& RT, int32_t n_active, int32_t layer,
                           int32_t* err, cudaStream_t s) {
  const int d8 = A.d / 8;
  const size_t smem = (size_t)A.half * 8 + (size_t)A.Hkv * 4;
  auto go = [&](auto kernel) {
    kernel<<<n_active, kThreads, smem, s>>>(A, G, S, RT, layer, err);
    return cudaGetLastError();
  };
  return d8 <= 4    ? go(append_qkv_kernel<T, 4>)
         : d8 <= 8  ? go(append_qkv_kernel<T, 8>)
         : d8 <= 16 ? go(append_qkv_kernel<T, 16>)
                    : go(append_qkv_kernel<T, 32>);
}

}  // namespace

cudaError_t launch_norm_rope(const RowArgs& A, int32_t dtype, int32_t n_rows, const int32_t* positions, void* k, void* v, cudaStream_t s) {
  RowsTo R{};
  R.n_rows = n_rows;
  R.positions = positions;
  R.k = k;
  R.v = v;
  return dtype == OKV_F32 ? run_rows<float, false>(A, R, s) : run_rows<__nv_bfloat16, false>(A, R, s);
}

cudaError_t launch_append_rows(const RowArgs& A, const Geom& G, int32_t n_requests, int32_t n_new, const int32_t* counts, const int32_t* len,
                               const int32_t* slot_block, void* pool, cudaStream_t s) {
  RowsTo R{};
  R.n_rows = n_requests;
  R.n_new = n_new;
  R.bs = G.bs;
  R.kb = G.kb;
  R.counts = counts;
  R.len = len;
  R.slot_block = slot_block;
  R.pool = pool;
  return G.dtype == OKV_F32 ? run_rows<float, true>(A, R, s) : run_rows<__nv_bfloat16, true>(A, R, s);
}

cudaError_t launch_append_qkv(const RowArgs& A, const Geom& G, const LayerState& S, const ReqTables& T, int32_t n_active, int32_t layer,
                              int32_t* err, cudaStream_t s) {
  if (n_active <= 0) return cudaSuccess;
  return G.dtype == OKV_F32 ? run_append_qkv<float>(A, G, S, T, n_active, layer, err, s)
                            : run_append_qkv<__nv_bfloat16>(A, G, S, T, n_active, layer, err, s);
}

cudaError_t launch_append_tree(const Geom& G, const LayerState& S, const ReqTables& T, int32_t n, int32_t layer, int32_t n_draft,
                               const void* k, const void* v, const Accepted& P, int32_t* arrivals, int32_t* err, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  const dim3 grid(n, G.Hkv);
  if (G.dtype == OKV_F32)
    append_tree_kernel<float><<<grid, 128, 0, s>>>(G, S, T, layer, n_draft, (const float*)k, (const float*)v, P, arrivals, err);
  else
    append_tree_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(G, S, T, layer, n_draft, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, P,
                                                          arrivals, err);
  return cudaGetLastError();
}

}  // namespace okv

extern "C" okv_status okv_norm_rope(int32_t n_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype, const void* qkv,
                                    int64_t row_stride, const int32_t* positions, const okv_rotary* rotary, void* q, void* k, void* v,
                                    void* stream) {
  using namespace okv;
  if (n_rows == 0) return OKV_OK;
  RowArgs A;
  if (n_rows < 0 || !positions || !row_args(rotary, q_heads, kv_heads, head_dim, dtype, qkv, row_stride, q, &A)) return OKV_EINVAL;
  if ((!q && !k && !v) || !aligned16(k) || !aligned16(v)) return OKV_EINVAL;
  if (okv_status st = check_stream(stream)) return st;
  return launch_norm_rope(A, dtype, n_rows, positions, k, v, (cudaStream_t)stream) == cudaSuccess ? OKV_OK : OKV_ECUDA;
}

extern "C" okv_status okv_append_qkv_static(int32_t n_requests, int32_t n_new, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                            int32_t block_size, int32_t slots, int32_t dtype, const void* qkv, int64_t row_stride,
                                            const int32_t* lengths, const int32_t* counts, const okv_rotary* rotary, void* pool,
                                            const int32_t* slot_block, void* q, void* stream) {
  using namespace okv;
  Geom G{};
  RowArgs A;
  if (!tree_geom(n_requests, q_heads, kv_heads, head_dim, block_size, slots, dtype, &G)) return OKV_EINVAL;
  if (n_new <= 0 || (int64_t)n_requests * n_new > INT32_MAX) return OKV_EINVAL;
  if (!row_args(rotary, q_heads, kv_heads, head_dim, dtype, qkv, row_stride, q, &A)) return OKV_EINVAL;
  if (!lengths || !pool || !aligned16(pool) || !slot_block) return OKV_EINVAL;
  if (okv_status st = check_stream(stream)) return st;
  return launch_append_rows(A, G, n_requests, n_new, counts, lengths, slot_block, pool, (cudaStream_t)stream) == cudaSuccess ? OKV_OK
                                                                                                                               : OKV_ECUDA;
}
