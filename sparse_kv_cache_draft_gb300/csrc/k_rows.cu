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
// inv_freq / 2 pi, as a 64-bit fraction of a turn, times the integer p modulo 2^64 is the phase with
// an error of p 2^-54 turns at most (6e-8 turns at position 2^31 and one radian per position).
//
// The rows move once in and once out. A head row is 8 elements on each of d / 8 lanes (a subgroup of
// the next power of two of lanes); a CTA takes the heads of a few tokens, four head rows in flight
// per subgroup, and computes the tokens' angles once, while the first loads are on their way.
#include <cuda_bf16.h>

#include "okv_tree.h"
#include "ptx.cuh"

namespace okv {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;  // head rows each subgroup loads before it computes

// 8 elements of a head row.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
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

// cos and sin of pos * f radians.
__device__ __forceinline__ void angle(float f, int32_t pos, float* c, float* s) {
  double turns = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  turns -= floor(turns);
  const uint64_t per = turns < 1.0 ? (uint64_t)(turns * 18446744073709551616.0) : 0;
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

// Norm and rotation of one head row over the LPG lanes of a subgroup; `sub` is the lane within it.
// Every lane of the warp calls it. cos / sin: the token's tables of `half` entries.
template <int LPG, typename T>
__device__ __forceinline__ void norm_turn(const RowArgs& A, float (&x)[8], const T* w, const float* cs, const float* sn, int sub, bool turn) {
  // the subgroups of a warp hold heads of different kinds: all of them reduce, the normed ones scale
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
  for (int off = LPG / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (w && sub * 8 < A.d) {
    const float r = 1.f / sqrtf(ss / (float)A.d + A.eps);
    Eight<T> wv;
    float wf[8];
    wv.load(w + sub * 8);
    wv.get(wf);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * wf[e];
  }
  const int step = A.half / 8;  // lanes between the two halves
  const bool low = sub < step, in = sub < 2 * step;
  if (A.interleaved) {
    if (turn && in) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = cs[sub * 4 + e], s = sn[sub * 4 + e];
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = a * c - b * s;
        x[2 * e + 1] = b * c + a * s;
      }
    }
  } else {
    const int lane = threadIdx.x & 31, other = in ? (low ? lane + step : lane - step) : lane;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], other);
    if (turn && in) {
      const int at = (low ? sub : sub - step) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = cs[at + e], s = low ? -sn[at + e] : sn[at + e];
        x[e] = x[e] * c + y[e] * s;
      }
    }
  }
}

// Where the rows of one launch come from and go to.
struct RowsTo {
  int32_t n_rows;              // norm_rope: rows; append: requests
  int32_t tok;                 // tokens of a CTA
  const int32_t* positions;    // norm_rope
  void *k, *v;                 // norm_rope: [rows][Hkv][d] or NULL
  // append
  int32_t n_new, bs, kb;
  const int32_t *counts, *len, *slot_block;
  void* pool;                  // [R][Hkv][kb][2][bs][d]
};

template <typename T, int LPG, bool APPEND>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowArgs A, const RowsTo R) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* cs = reinterpret_cast<float*>(smem);          // [tok][half]
  float* sn = cs + R.tok * A.half;                     // [tok][half]
  int32_t* slot_of = reinterpret_cast<int32_t*>(sn + R.tok * A.half);  // append: [Hkv][tok + 1]
  const int tid = threadIdx.x, sub = tid % LPG, group = tid / LPG;
  constexpr int kGroups = kThreads / LPG;
  const int32_t H = A.Hq + 2 * A.Hkv;

  int64_t row0;       // first row of the CTA
  int32_t n_tok;      // its rows
  int32_t r = 0, pos0 = 0, blk0 = 0;
  if (APPEND) {
    const int32_t per = (R.n_new + R.tok - 1) / R.tok;
    r = blockIdx.x / per;
    const int32_t t0 = (blockIdx.x - r * per) * R.tok;
    const int32_t cnt = R.counts ? min(max(R.counts[r], 0), R.n_new) : R.n_new;
    row0 = (int64_t)r * R.n_new + t0;
    n_tok = min(R.tok, cnt - t0);
    const int32_t len = R.len[r];
    if (n_tok <= 0 || len < 0 || len > INT32_MAX - R.n_new) return;  // positions stay within 31 bits
    pos0 = len + t0;
    blk0 = pos0 / R.bs;
  } else {
    row0 = (int64_t)blockIdx.x * R.tok;
    n_tok = min((int64_t)R.tok, R.n_rows - row0);
  }
  const int32_t items = n_tok * H;
  const bool on = sub * 8 < A.d;

  for (int32_t base = 0; base < items; base += kGroups * kInFlight) {
    Eight<T> raw[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int32_t i = base + u * kGroups + group;
      if (i < items && on) {
        const int32_t tk = i / H, h = i - tk * H;
        raw[u].load((const T*)A.qkv + (row0 + tk) * A.row_stride + (int64_t)h * A.d + sub * 8);
      }
    }
    if (base == 0) {
      const int32_t span = R.tok + 1;
      if (APPEND) {
        for (int32_t i = tid; i < A.Hkv * span; i += kThreads) slot_of[i] = INT32_MAX;
        __syncthreads();
        const int32_t last = (pos0 + n_tok - 1) / R.bs;
        const int32_t* sb = R.slot_block + (int64_t)r * A.Hkv * R.kb;
        for (int32_t i = tid; i < A.Hkv * R.kb; i += kThreads) {
          const int32_t b = sb[i];
          if (b >= blk0 && b <= last) atomicMin(&slot_of[i / R.kb * span + (b - blk0)], i % R.kb);
        }
      }
      for (int32_t i = tid; i < n_tok * A.half; i += kThreads) {
        const int32_t tk = i / A.half, f = i - tk * A.half;
        angle(A.inv_freq[f], APPEND ? pos0 + tk : R.positions[row0 + tk], &cs[i], &sn[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int32_t i = base + u * kGroups + group;
      const bool real = i < items;
      const int32_t tk = real ? i / H : 0, h = real ? i - tk * H : 0;
      const bool is_q = h < A.Hq, is_k = !is_q && h < A.Hq + A.Hkv;
      float x[8];
      if (real && on)
        raw[u].get(x);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      const T* w = (const T*)(is_q ? A.q_weight : is_k ? A.k_weight : nullptr);
      norm_turn<LPG, T>(A, x, w, cs + tk * A.half, sn + tk * A.half, sub, is_q || is_k);
      if (!real || !on) continue;
      if (is_q || is_k) raw[u].set(x);  // values pass as they are
      const int64_t row = row0 + tk;
      T* to = nullptr;
      if (is_q) {
        if (A.q) to = (T*)A.q + (row * A.Hq + h) * A.d;
      } else {
        const int32_t hk = is_k ? h - A.Hq : h - A.Hq - A.Hkv;
        if (APPEND) {
          const int32_t pos = pos0 + tk, b = pos / R.bs;
          const int32_t slot = slot_of[hk * (R.tok + 1) + (b - blk0)];
          if (slot != INT32_MAX)
            to = (T*)R.pool + (((((int64_t)r * A.Hkv + hk) * R.kb + slot) * 2 + (is_k ? 0 : 1)) * R.bs + (pos - b * R.bs)) * A.d;
        } else if (is_k ? R.k != nullptr : R.v != nullptr) {
          to = (T*)(is_k ? R.k : R.v) + (row * A.Hkv + hk) * A.d;
        }
      }
      if (!APPEND && R.positions[row] < 0) to = nullptr;
      if (to) raw[u].store(to + sub * 8);
    }
  }
}

template <typename T, bool APPEND>
cudaError_t run_rows(const RowArgs& A, RowsTo R, cudaStream_t s) {
  const int d8 = A.d / 8, lpg = d8 <= 4 ? 4 : d8 <= 8 ? 8 : d8 <= 16 ? 16 : 32;
  const int32_t H = A.Hq + 2 * A.Hkv, per_cta = kThreads / lpg * kInFlight;
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // tokens of a CTA: enough head rows for one full batch of loads, but no fewer CTAs than two per SM
  const int64_t tokens = APPEND ? (int64_t)R.n_rows * R.n_new : R.n_rows;
  int64_t tok = per_cta / H;
  if (tok > tokens / (2 * sms)) tok = tokens / (2 * sms);
  R.tok = (int32_t)(tok < 1 ? 1 : tok > 16 ? 16 : tok);
  const int64_t ctas = APPEND ? (int64_t)R.n_rows * ((R.n_new + R.tok - 1) / R.tok) : ((int64_t)R.n_rows + R.tok - 1) / R.tok;
  const size_t smem = (size_t)R.tok * A.half * 8 + (APPEND ? (size_t)A.Hkv * (R.tok + 1) * 4 : 0);
  if (ctas > INT32_MAX || smem > 48 * 1024) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)ctas, kThreads, smem, s>>>(A, R);
    return cudaGetLastError();
  };
  return lpg == 4    ? go(rows_kernel<T, 4, APPEND>)
         : lpg == 8  ? go(rows_kernel<T, 8, APPEND>)
         : lpg == 16 ? go(rows_kernel<T, 16, APPEND>)
                     : go(rows_kernel<T, 32, APPEND>);
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
  for (int32_t f = tid; f < A.half; f += kThreads) angle(A.inv_freq[f], pos, &cs[f], &sn[f]);
  __syncthreads();
  const int32_t H = A.Hq + 2 * A.Hkv;
  const T* from = (const T*)A.qkv + (int64_t)r * A.row_stride;
  const bool on = sub * 8 < A.d;
  for (int32_t base = 0; base < H; base += kGroups) {
    const int32_t h = base + group;
    const bool real = h < H && on, is_q = h < A.Hq, is_k = !is_q && h < A.Hq + A.Hkv;
    Eight<T> raw;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (real) {
      raw.load(from + (int64_t)h * A.d + sub * 8);
      raw.get(x);
    }
    norm_turn<LPG, T>(A, x, (const T*)(is_q ? A.q_weight : is_k ? A.k_weight : nullptr), cs, sn, sub, is_q || is_k);
    if (!real) continue;
    if (is_q || is_k) raw.set(x);
    if (is_q) {
      raw.store((T*)A.q + ((int64_t)r * A.Hq + h) * A.d + sub * 8);
    } else {
      const int32_t hk = is_k ? h - A.Hq : h - A.Hq - A.Hkv;
      put(G, places<T>(G, S, RT, layer, r, hk, pos, slot_of[hk], err), is_k ? 0 : 1, sub * 8, raw);
    }
  }
  __syncthreads();
  if (tid == 0) {
    S.len[r] = pos + 1;
    S.len_act[blockIdx.x] = pos + 1;
  }
}

// grid (n_active, Hkv), d / 8 lanes at work (the tokens of a block go through its summary in order).
// The last of a request's Hkv CTAs to finish (counted in arrivals[r], zero before and after)
// advances its length.
template <typename T>
__global__ void __launch_bounds__(128) append_tree_kernel(const Geom G, const LayerState S, const ReqTables RT, const int32_t layer, const int32_t n_draft,
                                                          const T* __restrict__ k, const T* __restrict__ v, const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ index, int32_t* __restrict__ arrivals, int32_t* err) {
  const int32_t r = RT.active[blockIdx.x], h = blockIdx.y, n = counts[r], tid = threadIdx.x;
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
      const int64_t at = (((int64_t)r * n_draft + index[(int64_t)r * n_draft + i]) * G.Hkv + h) * G.d + c;
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
    S.len_act[blockIdx.x] = pos0 + n;
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

cudaError_t launch_append_tree(const Geom& G, const LayerState& S, const ReqTables& T, int32_t n_active, int32_t layer, int32_t n_draft,
                               const void* k, const void* v, const int32_t* counts, const int32_t* index, int32_t* arrivals, int32_t* err,
                               cudaStream_t s) {
  if (n_active <= 0) return cudaSuccess;
  const dim3 grid(n_active, G.Hkv);
  if (G.dtype == OKV_F32)
    append_tree_kernel<float><<<grid, 128, 0, s>>>(G, S, T, layer, n_draft, (const float*)k, (const float*)v, counts, index, arrivals, err);
  else
    append_tree_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(G, S, T, layer, n_draft, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, counts,
                                                          index, arrivals, err);
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
