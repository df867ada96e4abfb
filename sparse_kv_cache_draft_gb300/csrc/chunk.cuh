// What the kernels of a chunk of new tokens share: who sees whom, a CTA's share of the rows, and the list of the slots that they see.
#pragma once

#include "okv_chunk.h"
#include "tiles.cuh"

namespace okv {

// New tokens of request r: 0 where its length leaves no room for n_new more positions.
__device__ __forceinline__ int32_t new_tokens(const ChunkArgs& A, int32_t r, int32_t len) {
  const int32_t n = A.counts ? A.counts[r] : A.T;  // on its way beside the length
  return len < 0 || (int64_t)len + A.T > INT32_MAX ? 0 : min(max(n, 0), A.T);
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

// One CTA's share of the work.
struct Span {
  int32_t r, h, part, parts, cnt, len;
  int32_t row0, rows;   // rows [row0, row0 + rows) of the unit's g * cnt
  int32_t p_lo, p_hi;   // positions of the first and the last of them
};

__device__ __forceinline__ void fill_span(const ChunkArgs& A, int32_t group_rows, Span& s) {
  s.len = A.len[s.r];
  s.cnt = new_tokens(A, s.r, s.len);
  s.rows = min(group_rows, s.cnt * A.G.g - s.row0);
  s.p_lo = s.len + s.row0 / A.G.g;
  s.p_hi = s.len + (s.row0 + s.rows - 1) / A.G.g;
}

// Element offset of row m's vector in q and out, [R][T][Hq][d], times 1 / d: its place in lse.
__device__ __forceinline__ int64_t row_place(const ChunkArgs& A, const Span& s, int32_t m) {
  const int32_t t = m / A.G.g, j = m - t * A.G.g;
  return ((int64_t)s.r * A.T + t) * A.G.Hq + s.h * A.G.g + j;
}
// The unit's slots that rows of the span see: `whole` of them, which all rows see whole, from the front of the list, the
// others from its back, the first positions of the first kBases of those beside it. By `warps` warps of which each takes
// a run of at most 256 slots: load, count, then place.
constexpr int kListWarps = 8, kBases = 128;
struct Listed {
  int32_t whole[kListWarps], some[kListWarps], base[kBases];
};
struct List {
  const uint16_t* at;  // [kb]
  const int32_t *base, *ids;
  int32_t kb, bs, whole, n;
  __device__ __forceinline__ int32_t slot(int32_t e) const { return at[e < whole ? e : kb - 1 - (e - whole)]; }
  // What position p sees of entry e, as bits of its tokens.
  __device__ __forceinline__ uint64_t seen(int32_t e, int32_t p, int32_t window, int32_t sinks) const {
    return e < whole ? first_bits(bs) : seen_of(first(e), p, bs, window, sinks);
  }
  __device__ __forceinline__ int32_t first(int32_t e) const { return e - whole < kBases ? base[e - whole] : ids[slot(e)] * bs; }  // e >= whole
};
struct Ids {
  int32_t b[8];  // of slots first + 32 u + lane
  int32_t per, first;
};
__device__ __forceinline__ Ids load_ids(const ChunkArgs& A, const Span& s, int warp, int warps) {
  const int32_t* sb = A.slot_block + ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb;
  Ids x;
  x.per = (A.G.kb + 32 * warps - 1) / (32 * warps);
  x.first = warp * x.per * 32;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int32_t i = x.first + u * 32 + (threadIdx.x & 31);
    x.b[u] = u < x.per && i < A.G.kb ? sb[i] : -1;
  }
  return x;
}
__device__ __forceinline__ void count_slots(const ChunkArgs& A, const Span& s, const Ids& x, int warp, Listed& L, uint32_t (&all)[8], uint32_t (&some)[8]) {
  int32_t nw = 0, ns = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (u >= x.per) break;
    const int32_t c = sight(x.b[u], A.G.bs, s.p_lo, s.p_hi, A.window, A.sinks);
    all[u] = __ballot_sync(0xffffffffu, c == 2);
    some[u] = __ballot_sync(0xffffffffu, c == 1);
    nw += __popc(all[u]);
    ns += __popc(some[u]);
  }
  if ((threadIdx.x & 31) == 0) L.whole[warp] = nw, L.some[warp] = ns;
}
__device__ __forceinline__ void place_slots(const ChunkArgs& A, const Ids& x, int warp, Listed& L, const uint32_t (&all)[8], const uint32_t (&some)[8],
                                            uint16_t* at) {
  const int lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  int32_t nw = 0, ns = 0;
  for (int w = 0; w < warp; ++w) nw += L.whole[w], ns += L.some[w];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (u >= x.per) break;
    const uint16_t slot = (uint16_t)(x.first + u * 32 + lane);
    if (all[u] >> lane & 1) at[nw + __popc(all[u] & below)] = slot;
    if (some[u] >> lane & 1) {
      const int32_t e = ns + __popc(some[u] & below);
      at[A.G.kb - 1 - e] = slot;
      if (e < kBases) L.base[e] = x.b[u] * A.G.bs;
    }
    nw += __popc(all[u]);
    ns += __popc(some[u]);
  }
}
__device__ __forceinline__ List make_list(const ChunkArgs& A, const Span& s, int warps, const Listed& L, const uint16_t* at) {
  List l{at, L.base, A.slot_block + ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb, A.G.kb, A.G.bs, 0, 0};
  for (int w = 0; w < warps; ++w) l.whole += L.whole[w], l.n += L.some[w];
  l.n += l.whole;
  return l;
}

// ---- a CTA's rows of the attention --------------------------------------------------------------------
// Where a CTA's share is; the longest groups of a unit, its last rows, come first. What needs the lengths is filled in below, so
// that they are on their way beside the slot table.
__device__ __forceinline__ Span make_span(const ChunkArgs& A, const Shape& P, int32_t group_rows) {
  Span s;
  const int32_t cluster = blockIdx.x / P.split, rank = blockIdx.x - cluster * P.split, wholes = P.whole / P.split;
  const bool whole = cluster < wholes;
  const int32_t item = whole ? (int32_t)blockIdx.x : P.whole + cluster - wholes;
  const int32_t ua = item / P.groups, group = P.groups - 1 - (item - ua * P.groups);
  s.part = whole ? 0 : rank;
  s.parts = whole ? 1 : P.split;
  s.r = ua / A.G.Hkv;
  s.h = ua - s.r * A.G.Hkv;
  s.row0 = group * group_rows;
  return s;
}

// Adds what the values that are not finite, of tokens in tiles that were masked, give to four outputs (dims c .. c + 3) of
// a row that sees them: they are zero in the products, where a weight of zero times them would reach rows that do not. (Arguments one by
// one: a struct whose address is taken is written to local memory by every thread, whether it comes here or not.)
template <typename T>
__device__ __noinline__ float4 not_finite_of(const ChunkArgs& A, int64_t unit, const uint16_t* at, const int32_t* base, int32_t whole, int32_t n, int32_t part,
                                              int32_t parts, int32_t spt, int32_t p, int32_t c) {
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const List L{at, base, A.slot_block + unit, A.G.kb, A.G.bs, whole, n};
  for (int32_t e = whole / spt * spt; e < n; ++e) {
    if (e / spt % parts != part) continue;
    const int32_t slot = L.slot(e);
    uint64_t bits = L.seen(e, p, A.window, A.sinks);
    const T* v = reinterpret_cast<const T*>(A.pool + (unit + slot) * A.G.block_bytes) + (int64_t)A.G.bs * A.G.d + c;
    while (bits) {
      const int32_t j = __ffsll((long long)bits) - 1;
      bits &= bits - 1;
      const float x = to_f(v[j * A.G.d]), y = to_f(v[j * A.G.d + 1]), z = to_f(v[j * A.G.d + 2]), w = to_f(v[j * A.G.d + 3]);
      if (!is_finite(x)) o.x += x;
      if (!is_finite(y)) o.y += y;
      if (!is_finite(z)) o.z += z;
      if (!is_finite(w)) o.w += w;
    }
  }
  return o;
}

// Merges the cluster's partials and writes outputs and sums. The first `threads` threads of every CTA of the cluster call it,
// the others cluster_sync twice.
template <typename T, typename F>
__device__ __forceinline__ void merge_chunk(const ChunkArgs& A, const Span& s, const Partial& P, int32_t xor_mask, int32_t threads, F more) {
  cluster_sync();
  more();
  merge_rows(s.part, s.parts, s.rows, A.G.d, P, xor_mask, threads, [&](int32_t row, int32_t c, float4 o, float M, float l) {
    const int64_t at = row_place(A, s, s.row0 + row);
    store4((T*)A.out + at * A.G.d + c * 4, o);
    if (c == 0 && A.lse) A.lse[at] = lse_of(M, l);
  });
  cluster_sync();  // no CTA leaves while another may still read its shared memory
}

// ---- launches ------------------------------------------------------------------------------------------
// Tiles that a group of rows has if no block is in two slots: of the slots there are, and of those that a window leaves it.
inline int32_t likely_tiles(const ChunkArgs& A, int32_t spt, int32_t group_tok) {
  const int64_t bs = A.G.bs, seen = ((int64_t)A.window + group_tok + bs - 1) / bs + 1 + ((int64_t)A.sinks + bs - 1) / bs;
  const int64_t slots = seen < A.G.kb ? seen : A.G.kb;
  return (int32_t)((slots + spt - 1) / spt);
}

}  // namespace okv
