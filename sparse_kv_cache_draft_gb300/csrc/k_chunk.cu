// Attention of a chunk of new tokens over a paged pool that holds them already.
//
// Token t of a request is at position p = length + t and sees the resident tokens at positions j <= p with
// p - j < window or j < sinks. For query head h of KV head k, over those tokens:
//   o_th = sum_j softmax_j(q_th . k_j / sqrt(d)) v_j,   lse_th = log sum_j exp(q_th . k_j / sqrt(d))
// zero and -infinity where there are none. The g T rows (t, head) of a unit (request, KV head) are taken in groups of up
// to 128 or 256; the slots that any row of a group sees are listed, those that all of its rows see whole first, so that
// few tiles of a group need a mask whatever the slots' order, and slots that no row sees are not read. Tiles are dealt
// to the CTAs of a cluster where there are too few groups to fill the GPU, as for drafted trees.
//
// Measured (32 / 8 heads of 128 dims, bf16): 4 requests x 1024 tokens with 64 / 8 heads behind 31K 2.58 to 2.80 ms, 1.55 to 1.68
// PFLOP/s, 0.80 to 0.87 of the measured rate, by the GPU's power; 2048 tokens behind 14K 348 to 370 us, 1.39 to 1.48 PFLOP/s (two
// rounds of 256 groups on 152 SMs); one token for 128 requests over 2048 resident ones 162 us, 0.97 of a copy's rate, 184 with the
// slots' weights; one token of one request 9.4 us.
#include <stddef.h>

#include "chunk.cuh"
#include "ring.h"

namespace okv {
namespace {

// ---- tensor cores: bf16 ------------------------------------------------------------------------------
//
// A CTA holds NW groups of 128 rows (a softmax warpgroup each) over the same tiles of tokens; a warp copies K and one V into a
// ring of buffers, and one thread issues the MMAs of all groups:
//   S = Q K^T   128 x tile, Q and K in shared memory, S in TMEM
//   O += P V    128 x d,    P in TMEM in the place of its S (bf16), V in shared memory, O in TMEM
// A thread takes a row's softmax; the running maximum moves when a row of the warp passes it by 2^8. Weights are rounded to bf16
// for the second product (half a step each), their sum is of the unrounded ones.
//
// Up to 128 rows (NW = 1) tiles are 64 tokens, S has two buffers and two CTAs share an SM: HBM is the limit. Beyond
// (NW = 2) tiles are 128 tokens with one S for each warpgroup, and while one has its products the other is at its softmax.
// What bounds it then: 32 MMAs of 64 cycles to a tile of both, and about 2600 cycles for it; the exponentials of 256 rows take
// 1024. A CTA's start and end are about 12 thousand cycles beside that.
//
// The steps that counted, 1024 tokens x 4 requests behind 31K, 64 / 8 heads: first version, with MMAs issued by a whole warp for
// each warpgroup in turns, 3657 us; registers of the other warps to the softmax's 3425; one elected thread, in whose branch the
// operands are known to be uniform, and the first weights beside the search for the maximum 2786; K and V waited for where
// they are used 2609; no spills 2532. 256 tokens x 16 requests over 2048 resident ones: 168 us, 148 by then, 122 with a warp for K and
// one for V, shorter lists and outputs by TMA.
//
// A tile is spt slots of the list. Slots that follow one another in the pool come in one copy for a line, others slot by
// slot. A slot's lines begin at a multiple of 128 bytes of shared memory: with lines of 64 bytes and an odd block
// size a line is left free behind each slot.
template <int NW>
struct Tiles {
  static constexpr int kTile = NW == 2 ? 128 : 64;
  static constexpr int kS = 128 / kTile;  // S buffers
};

constexpr int kMaxRing = 12;
struct MmaBars {
  uint64_t full[kMaxRing], empty[kMaxRing], q_full, s_full[2][2], p_full[2][2][2], pv_done[2][2], drain;
  Listed listed;
  uint32_t tmem;
  int32_t failed, bad, issued[2];  // issued: tiles whose keys, and whose values, were asked for
};

__host__ __device__ constexpr size_t mma_misc(int kb) { return sizeof(MmaBars) + ((size_t)kb * 2 + 15) / 16 * 16; }

// Up to 128 rows the weights that slots draw are summed on the way, where there is room: [entries][q_rows] sums of a row's weights over a
// slot's tokens, against the maximum of then, [tiles][q_rows], both of this CTA's tiles; with the final maxima and sums they are
// joined at the end. Where a slot is a multiple of eight columns of a tile, as the sums come by eight. At d 128, blocks of 16 and
// four heads to a key head there is room for 1024 slots for two tokens, 524 for four, 240 for eight, 92 for 16 and 20 for 32; beyond,
// a second launch reads the keys again (128 requests x 8 tokens: 209 us over 128 slots, 1079 over 256; without weights 167 and 308).
__host__ __device__ constexpr size_t drawn_bytes(int tiles, int spt, int q_rows) { return (size_t)tiles * (spt + 1) * q_rows * 4; }

struct ChunkMaps {
  CUtensorMap tile, slot, q, out;  // the pool by spt slots and by one, the queries, the outputs
};

// Whether line `row` of a tile holds a value that is not finite.
template <int D, int Tile>
__device__ __forceinline__ bool any_not_finite(const uint8_t* tile, int row) {
  uint32_t any = 0;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(tile + Lines<D, Tile>::piece(row, c));
    // an exponent of ones carries into the sign's place
    any |= ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) | ((x.z & 0x7F807F80u) + 0x00800080u) |
           ((x.w & 0x7F807F80u) + 0x00800080u);
  }
  return (any & 0x80008000u) != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Waits (bounded) for the copies that a warp, for values or for keys and the queries, started and that may be on their way still. Called where
// a block gives up, and not inlined: one token of 128 requests under a window takes 112.5 us, with this code in the kernel's 113.6.
template <int kS>
__device__ __noinline__ void land_copies(uint32_t full, uint32_t q_full, int32_t keys, int32_t values, bool v, int32_t ring) {
  using Order = RingOrder<kS>;
  const int32_t mine = v ? values : keys;
  for (int32_t i = max(0, mine - ring); i < mine; ++i) {
    const int32_t u = v ? Order::value(i) : Order::key(i);
    if (Order::may_be_on_its_way(u, ring, keys, values)) mbar_wait_timed(full + u % ring * 8, (uint32_t)(u / ring & 1));
  }
  if (!v) mbar_wait_timed(q_full, 0);
}

// Two warpgroups hold 128 scores to a thread, more registers than each thread of the block can have: the others, a whole
// warpgroup (one warp idle), give up what they do not need. 2 x 216 + 72 is what 3 x 168 were at the launch.
template <int NW>
constexpr int mma_threads() { return NW == 2 ? 384 : 224; }
constexpr int kUpRegs = 216, kDownRegs = 72;

template <int D, int NW, bool kDraw>
__global__ void __launch_bounds__(mma_threads<NW>(), D <= 128 && NW == 1 ? 2 : 1)
chunk_mma_kernel(const __grid_constant__ ChunkArgs A, const __grid_constant__ ChunkMaps M, const Shape shape, const int32_t rings, const int32_t q_tok,
                 const int32_t q_rows, const int32_t pitch, const int32_t most) {
  constexpr int kTile = Tiles<NW>::kTile, kS = Tiles<NW>::kS, kWords = kTile / 32;
  using L = Lines<D, kTile>;
  constexpr uint32_t kCols = D <= 128 ? 256 : 512;  // TMEM columns of a warpgroup: S in the first 128, O behind
  constexpr uint32_t kO = 128;
  constexpr uint32_t kDescQK = mma_desc_bf16(128, kTile, false), kDescPV = mma_desc_bf16(128, D, true);
  // barriers and list, then the tiles at a multiple of 1024: where the block's shared memory begins at one, nothing is lost (the
  // ring is at least four buffers either way, which a cluster's partials need)
  extern __shared__ __align__(1024) uint8_t smem_1024[];
  uint8_t* smem = smem_1024;
  MmaBars& B = *reinterpret_cast<MmaBars*>(smem);
  uint16_t* list_at = reinterpret_cast<uint16_t*>(&B + 1);                   // [kb]
  const int32_t spt = kTile / pitch;
  // kDraw: [most tiles][spt][q_rows] sums, [most tiles][q_rows] maxima
  float* drawn = reinterpret_cast<float*>(smem + mma_misc(A.G.kb));
  float* drawn_m = drawn + (size_t)most * spt * q_rows;
  const uint32_t begin = smem_u32(smem), behind = begin + (uint32_t)(mma_misc(A.G.kb) + (kDraw ? drawn_bytes(most, spt, q_rows) : 0));
  uint8_t* qs = smem + ((behind + 1023) / 1024 * 1024 - begin);              // [NW][chunks][q_rows][line]
  uint8_t* rs = qs + (size_t)NW * q_rows * D * 2;                            // [ring][chunks][tile][line]
  const int32_t ring = min(rings, (int32_t)((begin + dynamic_smem() - smem_u32(rs)) / L::kBuf));

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool is_copy = warp == NW * 4, is_mma = warp == NW * 4 + 1, is_copy_v = warp == NW * 4 + 2, is_soft = warp < NW * 4;
  const int32_t g = A.G.g, gr = q_tok * g;  // rows of a warpgroup: q_tok tokens, all heads of the group
  const int32_t bs = A.G.bs;
  const bool tails = spt * bs < kTile;      // lines of a tile that no token has
  const uint32_t ring0 = smem_u32(rs);
  if (is_copy) {  // what reads no memory of the call
    if (lane < 4) tma_prefetch_map(&M.tile + lane);
    constexpr int kP = offsetof(MmaBars, p_full) / 8;
    for (int i = lane; i < (int)(offsetof(MmaBars, listed) / 8); i += 32)
      mbar_init(smem_u32(B.full + i), i >= kP && i < kP + 8 ? 128 : 1);
    if (lane == 0) B.failed = B.bad = 0;
    fence_mbar_init();
  } else if (tails && is_soft) {
    // lines that no copy writes meet weights of zero
    for (int32_t i = tid; i < ring * (L::kBuf / 16); i += NW * 128) reinterpret_cast<uint4*>(rs)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
  }
  grid_wait();
  Span s = make_span(A, shape, NW * gr);
  Ids ids;
  if (is_soft) ids = load_ids(A, s, warp, NW * 4);
  fill_span(A, NW * gr, s);
  if (s.rows <= 0) {
    if (kDraw && s.part == 0)
      for (int32_t i = tid; i < A.G.kb; i += mma_threads<NW>()) {
        const int64_t at = ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb + i;
        A.weight_out[at] = A.weight ? A.weight[at] : 0.f;
      }
    return;
  }
  const int64_t unit = ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb;

  // Setup: the softmax warps list the slots, the copy warp starts the queries' copies.
  uint32_t all[8], some[8];
  if (is_copy) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      // rows (t, head of the group) of a box follow one another as the group's rows do; a box past the last
      // request's tokens is filled up with zeros
      const uint32_t q_bar = smem_u32(&B.q_full);
      const int32_t boxes = NW > 1 && s.rows > gr ? 2 : 1, tok0 = s.r * A.T;
      mbar_expect_tx(q_bar, (uint32_t)(boxes * gr * D * 2));
      for (int w = 0; w < boxes; ++w)
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_5d(smem_u32(qs) + (w * L::kChunks + c) * q_rows * L::kBytes, &M.q, q_bar, 0, c, 0, s.h, tok0 + s.row0 / g + w * q_tok);
    }
    __syncwarp();
  } else if (!is_soft) {
    if (is_mma) tmem_alloc(smem_u32(&B.tmem), kCols * NW);
  } else {
    count_slots(A, s, ids, warp, B.listed, all, some);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (is_soft) place_slots(A, ids, warp, B.listed, all, some, list_at);
  if (kDraw && is_soft && s.part == 0) {  // slots that no row sees draw nothing
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u >= ids.per) break;
      const int32_t i = ids.first + u * 32 + lane;
      if (i < A.G.kb && !((all[u] | some[u]) >> lane & 1)) A.weight_out[unit + i] = A.weight ? A.weight[unit + i] : 0.f;
    }
  }
  __syncthreads();
  grid_go();  // the TMEM is allocated
  const uint32_t tmem = __shfl_sync(0xffffffffu, B.tmem, 0);
  const List list = make_list(A, s, NW * 4, B.listed, list_at);
  const int32_t n = ((list.n + spt - 1) / spt - s.part + s.parts - 1) / s.parts;  // this CTA's tiles

  using Order = RingOrder<kS>;
  auto v_use = [](int32_t i) { return Order::value(i); };
  // ... by all lanes of a warp: what follows is by whole warps
  auto warp_wait = [&](uint64_t& bar, int32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_timed(smem_u32(&bar), (uint32_t)parity)) != 0;
  };
  auto fail = [&] { *(volatile int32_t*)&B.failed = 1; };

  if (!is_soft) {
    if (NW == 2) registers_down<kDownRegs>();
  }
  if (is_copy || is_copy_v) {
    // A warp for K and one for V. What they ask shared memory for, between MMAs that read it, takes them as long as a tile's
    // products: with one warp for both and slots in any order, it and not the copies set the pace.
    const bool v = is_copy_v;
    int32_t issued = 0;
    for (; issued < n; ++issued) {
      const int32_t i = issued, use = v ? v_use(i) : Order::key(i), b = use % ring;
      const int32_t e0 = (s.part + i * s.parts) * spt, ne = min(spt, list.n - e0), first = list.slot(e0);
      const int32_t my_slot = lane < ne * L::kChunks ? list.slot(e0 + lane / L::kChunks) : 0;
      bool run = ne == spt && pitch == bs;
      for (int32_t e = lane; e < ne; e += 32) run = run && list.slot(e0 + e) == first + e;
      run = __all_sync(0xffffffffu, run);
      if (use >= ring) {
        // with one S buffer K of tile j is free once S of tile j is there, V of tile j - 1 as well
        const int32_t j = (use - ring + 1) / 2;
        if (!(kS == 1 ? warp_wait(B.empty[j % kMaxRing], j / kMaxRing & 1) : warp_wait(B.empty[b], use / ring - 1 & 1))) {
          fail();
          break;
        }
      }
      const uint32_t to = ring0 + b * L::kBuf, bar = smem_u32(&B.full[b]);
      if (lane == 0) mbar_expect_tx(bar, (uint32_t)(ne * bs * D * 2));
      __syncwarp();
      if (run) {
        if (lane < L::kChunks) tma_load_5d(to + lane * L::kChunk, &M.tile, bar, 0, lane, 0, v ? 1 : 0, (int32_t)unit + first);
      } else {
        for (int32_t x = lane; x < ne * L::kChunks; x += 32) {
          const int32_t e = x / L::kChunks, c = x % L::kChunks, slot = x == lane ? my_slot : list.slot(e0 + e);
          tma_load_5d(to + c * L::kChunk + e * pitch * L::kBytes, &M.slot, bar, 0, c, 0, v ? 1 : 0, (int32_t)unit + slot);
        }
      }
    }
    if (lane == 0) B.issued[v] = issued;
    if (!v && n == 0) mbar_wait_timed(smem_u32(&B.q_full), 0);  // else the MMA warp waits for it
  } else if (is_mma) {
    // One warp for both warpgroups, in a fixed order: O of a tile and S of the next for one, then for the other. An answer from a
    // barrier takes 150 to 350 cycles while the tensor cores read shared memory, so each barrier is asked ahead, behind
    // MMAs that keep them busy meanwhile, and waited for only where it had not been passed by then. (A warp for
    // each warpgroup, in turns, left the tensor cores idle for 400 of 1980 cycles a turn.)
    if (elect_one()) {
      constexpr int kSteps = L::kElems / 16;
      constexpr uint32_t kHi = smem_desc_hi(L::kGroup, L::kSwizzle);
      const uint32_t q_chunk = (uint32_t)(q_rows * L::kBytes) >> 4;
      const uint32_t q_desc = smem_desc_lo(smem_u32(qs), 16), k_desc = smem_desc_lo(ring0, 16), v_desc = smem_desc_lo(ring0, L::kChunk);
      int32_t kb = 0, kp = 0, vb = v_use(0), vp = 0;  // buffers and parities of the next K and V
      bool ok = true;
      auto step = [&](int32_t& b, int32_t& parity, int32_t by) {
        b += by;
        if (b >= ring) b -= ring, parity ^= 1;
      };
      auto ask = [&](uint64_t& bar, int32_t parity) { return mbar_test(smem_u32(&bar), (uint32_t)parity); };
      auto passed = [&](bool asked, uint64_t& bar, int32_t parity) {
        if (!asked) ok = ok && mbar_wait_timed(smem_u32(&bar), (uint32_t)parity);
        tc_fence_after();
      };
      auto s_at = [&](int32_t i, int w) { return tmem + w * kCols + (kS == 2 ? (i & 1) * kTile : 0); };
      auto qk = [&](int32_t i, int w, int c0, int c1) {  // steps c0 .. c1 - 1 of S
        const uint32_t kd = k_desc + kb * (L::kBuf >> 4), qd = q_desc + w * L::kChunks * q_chunk;
#pragma unroll
        for (int c = c0; c < c1; ++c)
          mma_ss1(s_at(i, w), qd + c / kSteps * q_chunk + c % kSteps * 2, kd + c / kSteps * (L::kChunk >> 4) + c % kSteps * 2, kHi, kDescQK, c > 0);
        if (c1 < D / 16) return;
        mma_commit1(smem_u32(&B.s_full[w][i & 1]));
        if (kS == 2) mma_commit1(smem_u32(&B.empty[kb]));
        if (w == NW - 1) step(kb, kp, kS == 2 && i == 0 ? 1 : 2);
      };
      auto pv = [&](int32_t i, int w, int half) {
        const uint32_t vd = v_desc + vb * (L::kBuf >> 4);
#pragma unroll
        for (int c = half * 4; c < half * 4 + 4; ++c)
          mma_ts1(tmem + w * kCols + kO, s_at(i, w) + c * 8, vd + c * 2 * (L::kGroup >> 4), kHi, kDescPV, i > 0 || c > 0);
        if (half + 1 < kTile / 64) return;
        if (kS == 2 || i + 1 == n) mma_commit1(smem_u32(&B.pv_done[w][i & 1]));
        if (kS == 2) mma_commit1(smem_u32(&B.empty[vb]));
        if (w == NW - 1) step(vb, vp, 2);
      };
      constexpr int kHalf = D / 32;  // steps of half an S
      if (n > 0) {
        passed(false, B.q_full, 0);
        passed(false, B.full[kb], kp);
#pragma unroll
        for (int w = 0; w < NW; ++w)
          if (ok) qk(0, w, 0, D / 16);
        if (ok) passed(false, B.full[vb], vp);
      }
      if (kS == 2) {
        bool k_there = false;
        for (int32_t i = 0; i < n && ok; ++i) {
          if (i + 1 < n) {
            passed(k_there, B.full[kb], kp);
            if (ok) qk(i + 1, 0, 0, D / 16);
          }
          passed(ask(B.p_full[0][i & 1][0], (i >> 1) & 1), B.p_full[0][i & 1][0], (i >> 1) & 1);
          if (!ok) break;
          pv(i, 0, 0);
          if (i + 1 < n) {
            passed(ask(B.full[vb], vp), B.full[vb], vp);
            k_there = i + 2 < n && ask(B.full[kb], kp);
          }
        }
      } else {
        bool next = false, v_there = true, k_there = false;  // what was asked last
        for (int32_t i = 0; i < n && ok; ++i) {
          const int32_t parity = (i >> 1) & 1;
          const bool more = i + 1 < n;
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            uint64_t(&p)[2] = B.p_full[w][i & 1];
            if (w == 0 && i > 0) passed(v_there, B.full[vb], vp);
            passed(next, p[0], parity);
            if (!ok) break;
            const bool there = ask(p[1], parity);
            pv(i, w, 0);
            passed(there, p[1], parity);
            if (!ok) break;
            pv(i, w, 1);
            next = false;
            if (!more) continue;
            // S takes the place of the P just used: the products run in order
            if (w == 0) passed(k_there, B.full[kb], kp);
            if (!ok) break;
            qk(i + 1, w, 0, kHalf);
            if (w + 1 < NW) {
              next = ask(B.p_full[w + 1][i & 1][0], parity);
            } else {
              int32_t k2 = kb, kp2 = kp;
              step(k2, kp2, 2);
              v_there = ask(B.full[vb], vp);
              k_there = i + 2 < n && ask(B.full[k2], kp2);
              next = ask(B.p_full[0][(i + 1) & 1][0], ((i + 1) >> 1) & 1);
            }
            qk(i + 1, w, kHalf, D / 16);
          }
        }
      }
      if (!ok) {
        fail();
        mma_commit1(smem_u32(&B.drain));
        mbar_wait_timed(smem_u32(&B.drain), 0);
      }
    }
    __syncwarp();
  }
  if (!is_soft) {  // the others' ends: see below
    __syncthreads();
    if (*(volatile int32_t*)&B.failed != 0) {
      // A wait ran out somewhere: copies that nobody came to wait for land before the shared memory is used for anything else.
      if (is_copy || is_copy_v) land_copies<kS>(smem_u32(B.full), smem_u32(&B.q_full), B.issued[0], B.issued[1], is_copy_v, ring);
      __syncthreads();
    }
    if (s.parts > 1) cluster_sync(), cluster_sync();
    __syncthreads();
    if (is_mma) {
      tc_fence_after();
      tmem_free(tmem, kCols * NW);
    }
  } else {
    if (NW == 2) registers_up<kUpRegs>();
    float m_run = -INFINITY, l_run = 0.f;
    const int w = warp >> 2, row = tid & 127, wrow = w * gr + row;
    const bool real = row < gr && wrow < s.rows, active = (warp & 3) * 32 < min(gr, s.rows - w * gr);
    const uint32_t my = tmem + w * kCols + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the TMEM lanes
    const float scale = kLog2e * rsqrtf((float)D);
    const int32_t p = s.len + (s.row0 + wrow) / g;
    if (!real) m_run = INFINITY;  // no vote below: what such a row holds moves no other row's maximum
    float neg = real ? 0.f : -INFINITY;  // -m_run, 0 where there is none yet
    uint32_t ends[kWords];        // the places of a tile that a token has
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const int32_t c = 32 * u + lane;
      ends[u] = tails ? __ballot_sync(0xffffffffu, c / pitch < spt && c % pitch < bs) : ~0u;
    }
    uint32_t closes = 0;          // bit k: columns 8 k .. 8 k + 7 of a tile are the last of a slot
    if (kDraw)
      for (int k = 0; k < 8; ++k) closes |= (uint32_t)((k + 1) * 8 % pitch == 0) << k;
    for (int32_t i = 0; i < n; ++i) {
      const int32_t e0 = (s.part + i * s.parts) * spt;
      const bool part_seen = e0 + spt > list.whole;  // who sees what differs, or the tile is not full
      uint32_t vis[kWords];
#pragma unroll
      for (int u = 0; u < kWords; ++u) vis[u] = ends[u];
      if (part_seen) {
        const int32_t ne = min(spt, list.n - e0);
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int32_t k0 = 0; k0 < ne; k0 += 32) {
          // the entries' first positions, one to a lane: shared memory answers late beside the MMAs. Of an entry that all see
          // whole, one that all do.
          const int32_t mine = k0 + lane < ne && e0 + k0 + lane >= list.whole ? list.first(e0 + k0 + lane) : INT32_MIN;
#pragma unroll 4
          for (int32_t k = k0; k < min(ne, k0 + 32); ++k) {
            const int32_t base = __shfl_sync(0xffffffffu, mine, k - k0), at = k * pitch;
            const uint64_t bits = base == INT32_MIN ? first_bits(bs) : seen_of(base, p, bs, A.window, A.sinks);
            if (at < 64) {
              lo |= bits << at;
              if (at) hi |= bits >> (64 - at);
            } else {
              hi |= bits << (at - 64);
            }
          }
        }
        const uint64_t both[2] = {lo, hi};
#pragma unroll
        for (int u = 0; u < kWords; ++u) vis[u] = (uint32_t)(both[u / 2] >> 32 * (u & 1));
        // Values that are not finite meet weights of zero: they are zero in the products. The first warpgroup sees to it, whose
        // product is the first of both; a line is one thread's.
        if (w == 0) {
          if (!warp_wait(B.full[v_use(i) % ring], (v_use(i) / ring) & 1)) {
            fail();
            break;
          }
          uint8_t* v = rs + (size_t)(v_use(i) % ring) * L::kBuf;
          const bool any = row < kTile && any_not_finite<D, kTile>(v, row);
          if (__any_sync(0xffffffffu, any)) {
            if (any) {
              const int32_t k = row / pitch, e = e0 + k;
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) {
                uint4* x = reinterpret_cast<uint4*>(v + L::piece(row, c));
                uint4 y = *x;
                if (clean(y)) *x = y;
              }
              // a token that some row may see?
              if (k < ne && (e < list.whole || list.first(e) <= s.p_hi - (row - k * pitch))) *(volatile int32_t*)&B.bad = 1;
            }
            __syncwarp();
            fence_proxy_async();
          }
        }
      }
      if (!warp_wait(B.s_full[w][i & 1], (i >> 1) & 1)) {
        fail();
        break;
      }
      if (kS == 1 && w == NW - 1 && row == 0) mbar_arrive(smem_u32(&B.empty[i % kMaxRing]));
      // With two S buffers, S of tile i follows O of tile i - 2, so this passes at once; it keeps each barrier's
      // waits in step with its phases, where tile i - 1's below is waited for only now and then
      if (kS == 2 && i > 1 && !warp_wait(B.pv_done[w][i & 1], ((i - 2) >> 1) & 1)) {
        fail();
        break;
      }
      tc_fence_after();
      bool lost = false;
      const uint32_t st = my + (kS == 2 ? (i & 1) * kTile : 0);
      uint32_t a[kWords][32], pk[32];
      float2 sums[kDraw ? 8 : 2];  // of the weights; with kDraw of eight columns each
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      // scores of 64 columns as they count
      auto mask = [&](int u0, int u1) {
        if (!part_seen && !tails) return;
#pragma unroll
        for (int u = u0; u < u1; ++u)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(vis[u] >> e & 1)) a[u][e] = 0xFF800000u;
      };
      auto maxima = [&](int e) {
#pragma unroll
        for (int u = 0; u < kWords; ++u) mx[u] = max3(mx[u], __uint_as_float(a[u][2 * e]), __uint_as_float(a[u][2 * e + 1]));
      };
      // the weights of 64 columns against m_run, and, where asked for, the maximum of as many
      auto weights = [&](int half, int with_max) {
        const float2 scale2 = make_float2(scale, scale), neg2 = make_float2(neg, neg);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t *x0 = &a[2 * half][2 * e], *y0 = &a[2 * half + 1][2 * e];
          float2 x = fma2(make_float2(__uint_as_float(x0[0]), __uint_as_float(x0[1])), scale2, neg2);
          float2 y = fma2(make_float2(__uint_as_float(y0[0]), __uint_as_float(y0[1])), scale2, neg2);
          x = make_float2(ex2(x.x), ex2(x.y));
          y = make_float2(ex2(y.x), ex2(y.y));
          float2 &sx = sums[kDraw ? e / 4 : 0], &sy = sums[kDraw ? 4 + e / 4 : 1];
          sx = add2(sx, x);
          sy = add2(sy, y);
          pk[e] = pack2(x.x, x.y);
          pk[16 + e] = pack2(y.x, y.y);
          if (with_max) maxima(e);
        }
      };
      auto no_sums = [&] {
#pragma unroll
        for (float2& x : sums) x = make_float2(0.f, 0.f);
      };
      no_sums();
      if (active) {
#pragma unroll
        for (int u = 0; u < kWords; ++u) tmem_ld32(a[u], st + 32 * u);
#pragma unroll
        for (int u = 0; u < kWords; ++u) tmem_wait_ld(a[u]);
        mask(0, kWords);
        // The maximum moves in few tiles: the first weights are taken against the old one beside the search for the
        // new one, and again where it moves (S is still there).
        if (i > 0) {
          weights(0, 1);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) maxima(e);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        if (__any_sync(0xffffffffu, top > m_run + 8.f) || i == 0) {
          const float mn = real ? larger_max(m_run, top) : m_run;  // of every row of the warp: the next vote is then far off
          const float f = m_run == mn ? 1.f : ex2(m_run - mn);
          m_run = mn;
          l_run *= f;
          neg = m_run == -INFINITY ? 0.f : -m_run;
          if (i > 0) {
            // O has the products of tile i - 1; with one S buffer those came before S of this tile
            if (kS == 2) lost = !warp_wait(B.pv_done[w][(i - 1) & 1], ((i - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D; k += 16) {
              uint32_t o[16];
              tmem_ld16(o, my + kO + k);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(my + kO + k, o);
            }
          }
          tmem_ld32(a[0], st);
          tmem_ld32(a[1], st + 32);
          tmem_wait_ld(a[0]);
          tmem_wait_ld(a[1]);
          mask(0, 2);
          no_sums();
          weights(0, 0);
        }
      }
      if (lost) {
        fail();
        break;
      }
#pragma unroll
      for (int half = 0; half < kWords / 2; ++half) {
        if (active) {
          if (half) weights(half, 0);
          tmem_st32(st + 32 * half, pk);  // over scores that have been read
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&B.p_full[w][i & 1][half]));
      }
      if constexpr (kDraw) {
        // sums of slots, behind the product's start; a slot is eight columns or a multiple of them
        float all = 0.f, sum = 0.f;
        float* to = drawn + (size_t)i * spt * q_rows + row;
        const bool keep = active && real;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x = sums[k].x + sums[k].y;
          all += x;
          sum += x;
          if (!(closes >> k & 1)) continue;
          if (keep) *to = sum;
          to += q_rows;
          sum = 0.f;
        }
        l_run += all;
        if (keep) drawn_m[i * q_rows + row] = m_run;
      } else {
        sums[0] = add2(sums[0], sums[1]);
        l_run += sums[0].x + sums[0].y;
      }
    }
    // with one S buffer the last tile's alone is counted there
    if (n > 0 && !warp_wait(B.pv_done[w][(n - 1) & 1], kS == 2 ? ((n - 1) >> 1) & 1 : 0)) fail();
    tc_fence_after();
    __syncthreads();  // every product done: the ring and Q become the outputs' and the cluster's
    const bool failed = *(volatile int32_t*)&B.failed != 0;
    if (failed) {
      __syncthreads();  // for the copies, see above
      const RowSums end = sums_at_end(true, m_run, l_run);
      m_run = end.m, l_run = end.l;
    }
    const bool bad = B.bad && real && l_run != 0.f;
    const int32_t rows = min(gr, s.rows - w * gr) - (warp & 3) * 32;  // of this warp
    auto extra = [&](uint32_t (&o)[32], int c) {
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 x = not_finite_of<__nv_bfloat16>(A, unit, list.at, list.base, list.whole, list.n, s.part, s.parts, spt, p, c + e);
        o[e] = __float_as_uint(__uint_as_float(o[e]) + x.x);
        o[e + 1] = __float_as_uint(__uint_as_float(o[e + 1]) + x.y);
        o[e + 2] = __float_as_uint(__uint_as_float(o[e + 2]) + x.z);
        o[e + 3] = __float_as_uint(__uint_as_float(o[e + 3]) + x.w);
      }
    };
    if (rows > 0 && s.parts == 1) {
      // through shared memory (in the place of the queries), to write whole lines: a warpgroup's by TMA as the queries came, or,
      // where some of its rows are not the request's, a warp's row by row
      constexpr int kPieces = D / 8, kXor = kPieces % 8 ? 3 : 7;  // pieces of eight rows on different banks
      constexpr int kAtOnce = NW == 2 && D % 64 == 0 ? 64 : 32;
      const bool full = (w + 1) * gr <= s.rows;
      uint8_t* own = qs + (size_t)w * q_rows * D * 2;
      uint8_t* mine = own + (size_t)(warp & 3) * 32 * D * 2;
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      if (real && A.lse) A.lse[row_place(A, s, s.row0 + wrow)] = lse_of(m_run, l_run);
      auto store = [&](int chunk) {  // a line of the rows, on its way while the next one is made
        fence_proxy_async();
        asm volatile("bar.sync %0, %1;" ::"r"(w + 1), "r"((gr + 31) / 32 * 32) : "memory");  // the warps that have rows
        if (row == 0)
          tma_store_5d(&M.out, smem_u32(own) + chunk * q_rows * L::kBytes, 0, chunk, 0, s.h, s.r * A.T + s.row0 / g + w * q_tok);
      };
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += kAtOnce) {
        uint32_t o[kAtOnce / 32][32];
        __syncwarp();
        if (n > 0) {
#pragma unroll
          for (int u = 0; u < kAtOnce / 32; ++u) tmem_ld32(o[u], my + kO + c0 + 32 * u);
#pragma unroll
          for (int u = 0; u < kAtOnce / 32; ++u) tmem_wait_ld(o[u]);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce / 32; ++u) {
          if (!real) break;
          const int c = c0 + 32 * u;
          if (l_run == 0.f) {  // no weights (but infinite values, perhaps)
#pragma unroll
            for (int e = 0; e < 32; ++e) o[u][e] = 0;
          }
          if (bad) extra(o[u], c);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[u][e + k]) * inv;
            const int piece = (c + e) / 8;
            uint8_t* to = full ? own + (piece / (L::kBytes / 16)) * (q_rows * L::kBytes) + L::at(row, piece % (L::kBytes / 16))
                               : mine + ((size_t)lane * kPieces + (piece ^ (lane & kXor))) * 16;
            *reinterpret_cast<uint4*>(to) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
          }
        }
        if (full && (c0 + kAtOnce) % L::kElems == 0) store(c0 / L::kElems);
      }
      if (full && row == 0) bulk_stores_read();
      __syncwarp();
      const uint32_t per_g = (65536 + g - 1) / g;  // m * per_g >> 16 is m / g for the rows of a group
      const int32_t m0 = w * gr + (warp & 3) * 32;
      __nv_bfloat16* base = (__nv_bfloat16*)A.out + row_place(A, s, s.row0) * D;  // row0 is the first head of a token
#pragma unroll 4
      for (int e = full ? 32 * kPieces : lane; e < min(rows, 32) * kPieces; e += 32) {
        const int r = e / kPieces, c = e - r * kPieces;
        const uint32_t m = m0 + r, t = m * per_g >> 16;
        const uint4 x = *reinterpret_cast<const uint4*>(mine + ((size_t)r * kPieces + (c ^ (r & kXor))) * 16);
        *reinterpret_cast<uint4*>(base + ((int64_t)t * A.G.Hq + (m - t * g)) * D + c * 8) = x;
      }
    } else if (rows > 0 && s.parts > 1) {
      float* ml = reinterpret_cast<float*>(qs);
      if (real) {
        ml[wrow] = m_run;
        ml[NW * q_rows + wrow] = l_run;
      }
      if (n > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(o, my + kO + c);
          tmem_wait_ld(o);
          if (!real) continue;
          if (bad) extra(o, c);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(rs + part_chunk(wrow, (c + e) / 4, D, 7)) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
    }
    const Partial mine_of{smem_u32(rs), smem_u32(qs), smem_u32(qs) + (uint32_t)(NW * q_rows * 4)};
    auto join = [&] {
      // what a row's weights of a tile are worth by now, then the slots' sums over the rows
      if (real) {
        float m = m_run, l = l_run;
        if (s.parts > 1) {
          m = -INFINITY, l = 0.f;
          for (int32_t k = 0; k < s.parts; ++k) m = fmaxf(m, ld_cluster(cluster_map(mine_of.m + row * 4, k)));
          for (int32_t k = 0; k < s.parts; ++k) {
            const float mk = ld_cluster(cluster_map(mine_of.m + row * 4, k)), lk = ld_cluster(cluster_map(mine_of.l + row * 4, k));
            if (lk != 0.f) l += (mk == -INFINITY ? 1.f : ex2(mk - m)) * lk;  // scores that are all NaN have a sum, but no maximum
          }
        }
        for (int32_t i = 0; i < n; ++i) {
          float& at = drawn_m[i * q_rows + row];
          // without a maximum the weights are zeros, or not numbers, as their sum then; an infinite sum leaves zero of finite weights,
          // and no number of the infinite ones
          at = l == 0.f ? 0.f : at == -INFINITY ? (l == l ? 0.f : l) : ex2(at - m) / l;
        }
      }
      asm volatile("bar.sync 9, 128;" ::: "memory");
      for (int32_t x = row; x < n * spt; x += 128) {
        const int32_t i = x / spt, e = (s.part + i * s.parts) * spt + x - i * spt;
        if (e >= list.n) break;
        float sum = 0.f;
        for (int32_t k = 0; k < s.rows; ++k) {
          const float f = drawn_m[i * q_rows + k];
          // a row whose sum is not a number makes all that it sees so, and nothing else
          if (f == f || list.seen(e, s.len + k / g, A.window, A.sinks)) sum = fmaf(drawn[(size_t)x * q_rows + k], f, sum);
        }
        const int64_t at = unit + list.slot(e);
        A.weight_out[at] = (A.weight ? A.weight[at] : 0.f) + (failed ? 0.f : sum);
      }
    };
    if (kDraw && s.parts == 1) join();
    if (s.parts > 1) merge_chunk<__nv_bfloat16>(A, s, mine_of, 7, NW * 128, [&] { if (kDraw) join(); });
    tc_fence_before();
    __syncthreads();
  }
}

// ---- launches ----------------------------------------------------------------------------------------------

// Those of the drafted trees. They were not fitted for these kernels: a start and end of the wide one are 4.6 of its tiles, not one.
constexpr Costs kMmaCosts{5.5, 6, 1}, kMmaCostsWide{1, 6, 1};

// Maps of 5 dims over lines and chunks: the pool as [slots][K, V][tokens], a box of one chunk of the tokens of spt slots
// or of one; the queries and outputs as [tokens][KV heads][group], a box of q_tok tokens of a KV head.
template <int D, int Tile>
cudaError_t make_maps(const ChunkArgs& A, int32_t spt, int32_t q_tok, ChunkMaps* m) {
  using L = Lines<D, Tile>;
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
  const cuuint64_t g = A.G.g, hkv = A.G.Hkv, bs = A.G.bs, slots = (cuuint64_t)A.pool_rows;
  const bool ok = encode(&m->tile, A.pool, {bs, 2, slots}, {token, half, 2 * half}, {(cuuint32_t)bs, 1, (cuuint32_t)spt}) &&
                  encode(&m->slot, A.pool, {bs, 2, slots}, {token, half, 2 * half}, {(cuuint32_t)bs, 1, 1}) &&
                  encode(&m->q, A.q, {g, hkv, all}, {token, token * g, token * g * hkv}, {(cuuint32_t)g, 1, (cuuint32_t)q_tok}) &&
                  encode(&m->out, A.out, {g, hkv, all}, {token, token * g, token * g * hkv}, {(cuuint32_t)g, 1, (cuuint32_t)q_tok});
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int NW, bool kDraw = false>
cudaError_t run_mma(const ChunkArgs& A, bool* drawn, cudaStream_t s) {
  constexpr int kTile = Tiles<NW>::kTile;
  using L = Lines<D, kTile>;
  const int32_t pitch = A.G.bs * L::kBytes % 128 ? A.G.bs + 1 : A.G.bs, spt = kTile / pitch;
  // a warpgroup's rows: all heads of as many tokens as fit 128
  const int32_t q_tok = A.T < 128 / A.G.g ? A.T : 128 / A.G.g, gr = q_tok * A.G.g, q_rows = (gr + 7) / 8 * 8;
  const int32_t groups = (A.T + NW * q_tok - 1) / (NW * q_tok);
  // Two CTAs on an SM where TMEM allows (2 x 256 columns), else one: the ring takes what is left of
  // that share of the shared memory. It is never so small that a third CTA, or one of 256 columns beside one of 512, could
  // come to wait for TMEM (two clusters that each hold what the other waits for would wait for ever).
  const bool two = D <= 128 && NW == 1;
  // the slots' sums, where the ring keeps the four buffers that it needs: of all slots, which may all hold the same block
  const int32_t most = (A.G.kb + spt - 1) / spt;
  const size_t share = two ? 115712 : kMaxSmem, tiles0 = (size_t)NW * q_rows * D * 2, sums = kDraw ? drawn_bytes(most, spt, q_rows) : 0;
  if constexpr (NW == 1 && !kDraw) {
    const size_t all = drawn_bytes(most, spt, q_rows) + mma_misc(A.G.kb) + 2048 + tiles0 + 4 * L::kBuf;
    if (A.weight_out && groups == 1 && pitch % 8 == 0 && all <= share) return run_mma<D, NW, true>(A, drawn, s);
  }
  *drawn = kDraw;
  const size_t rest = (mma_misc(A.G.kb) + sums + 1023) / 1024 * 1024 + tiles0;
  int32_t ring = (int32_t)((share - rest) / L::kBuf);
  if (ring > kMaxRing) ring = kMaxRing;
  size_t smem = rest + (size_t)ring * L::kBuf + 1024;
  if (smem > share) smem = share;
  const size_t third = 233472 / 3, least = two ? third : 2 * third;
  if (smem < least) smem = least;
  const int64_t items = (int64_t)A.G.R * A.G.Hkv * groups;
  const int32_t per_sm = two ? 2 : 1;
  const Shape shape = pick_shape(items, groups, per_sm, likely_tiles(A, spt, NW * q_tok), NW == 1 ? kMmaCosts : kMmaCostsWide,
                                 cluster_room(mma_threads<NW>(), per_sm));
  ChunkMaps maps;
  if (cudaError_t e = make_maps<D, kTile>(A, spt, q_tok, &maps)) return e;
  return launch_cluster(chunk_mma_kernel<D, NW, kDraw>, items, shape, mma_threads<NW>(), smem, s, A, maps, shape, ring, q_tok, q_rows, pitch, most);
}

// *drawn: whether the slots' weights are summed on the way.
cudaError_t run_mma_d(const ChunkArgs& A, bool* drawn, cudaStream_t s) {
  const bool wide = (int64_t)A.T * A.G.g > 128;
  switch (A.G.d) {
    case 32: return wide ? run_mma<32, 2>(A, drawn, s) : run_mma<32, 1>(A, drawn, s);
    case 64: return wide ? run_mma<64, 2>(A, drawn, s) : run_mma<64, 1>(A, drawn, s);
    case 96: return wide ? run_mma<96, 2>(A, drawn, s) : run_mma<96, 1>(A, drawn, s);
    case 128: return wide ? run_mma<128, 2>(A, drawn, s) : run_mma<128, 1>(A, drawn, s);
    case 160: return run_mma<160, 1>(A, drawn, s);
    case 192: return run_mma<192, 1>(A, drawn, s);
    case 224: return run_mma<224, 1>(A, drawn, s);
    default: return run_mma<256, 1>(A, drawn, s);
  }
}

}  // namespace

cudaError_t launch_attend_chunk(const ChunkArgs& A, cudaStream_t s) {
  bool drawn = false;
  const cudaError_t e = A.G.dtype == OKV_F32 ? launch_chunk_f32(A, s) : run_mma_d(A, &drawn, s);
  return e != cudaSuccess || drawn || !A.weight_out ? e : launch_weigh_chunk(A, s);
}

}  // namespace okv

extern "C" okv_status okv_attend_chunk_static(int32_t n_requests, int32_t n_new, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                              int32_t block_size, int32_t slots, int32_t dtype, const void* pool, const int32_t* slot_block,
                                              const int32_t* lengths, const int32_t* counts, int32_t window, int32_t sinks, const void* q,
                                              void* out, float* lse, const float* weight, float* weight_out, void* stream) {
  using namespace okv;
  Geom G{};
  if (!tree_geom(n_requests, q_heads, kv_heads, head_dim, block_size, slots, dtype, &G)) return OKV_EINVAL;
  // rows of a unit are counted in 32 bits, those of the last group and of the one behind it, up to 256 each, among them
  if (n_new <= 0 || (int64_t)n_requests * kv_heads * n_new > INT32_MAX || (int64_t)n_new * G.g > INT32_MAX - 512) return OKV_EINVAL;
  if (window < 0 || sinks < 0) return OKV_EINVAL;
  if (!pool || !slot_block || !lengths || !q || !out || (weight_out && !lse) || (weight && !weight_out)) return OKV_EINVAL;
  if (!aligned16(pool) || !aligned16(q) || !aligned16(out)) return OKV_EINVAL;
  if (okv_status st = check_stream(stream)) return st;
  ChunkArgs A{};
  A.G = G;
  A.T = n_new;
  A.pool = (const uint8_t*)pool;
  A.slot_block = slot_block;
  A.len = lengths;
  A.counts = counts;
  A.q = q;
  A.out = out;
  A.lse = lse;
  A.window = window ? window : INT32_MAX;
  A.sinks = sinks;
  A.weight = weight;
  A.weight_out = weight_out;
  A.pool_rows = (int64_t)n_requests * kv_heads * slots;
  return launch_attend_chunk(A, (cudaStream_t)stream) == cudaSuccess ? OKV_OK : OKV_ECUDA;
}
