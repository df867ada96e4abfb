// The attention weight that each slot of a paged pool draws from a chunk of new tokens.
//
//   weight_out[s] = weight[s] + sum over the rows (t, head) of the unit and the tokens j of slot s that the row sees of
//                   exp(q . k_j / sqrt(d) - lse)
// with the sums lse that the attention of the chunk (k_chunk.cu) left. A CTA takes some of the unit's slots and every row
// that sees any of them, so that a slot's sum is one CTA's, in one order, and nothing is added by atomics.
//
// Measured: 8 requests of up to 512 new tokens, 32 / 8 heads of 128 dims, 4096 tokens in the pool, 136 us; exponentials and
// tensor cores are each busy 35% of the time.
#include <stddef.h>

#include <type_traits>

#include "chunk.cuh"

namespace okv {
namespace {

// One CTA's share: a tile of slots of a unit.
struct Site {
  int32_t r, h, cnt, len;
  int32_t slot0, slots;  // of the unit
};
__device__ __forceinline__ Site make_site(const ChunkArgs& A, int32_t spt, int32_t tiles) {
  Site s;
  const int32_t ua = blockIdx.x / tiles;
  s.slot0 = (blockIdx.x - ua * tiles) * spt;
  s.slots = min(spt, A.G.kb - s.slot0);
  s.r = ua / A.G.Hkv;
  s.h = ua - s.r * A.G.Hkv;
  s.len = A.len[s.r];
  s.cnt = new_tokens(A, s.r, s.len);
  return s;
}

// Rows [lo, hi) of the unit's g cnt that see token `off` of block b.
struct Rows {
  int32_t lo, hi;
};
__device__ __forceinline__ Rows rows_of(const ChunkArgs& A, const Site& s, int32_t b, int32_t off) {
  const int64_t t0 = (int64_t)b * A.G.bs + off - s.len;  // the first token that is not before it
  if (b < 0 || t0 >= s.cnt) return {0, 0};
  int64_t t1 = t0 + s.len < A.sinks ? s.cnt : t0 + A.window;
  if (t1 > s.cnt) t1 = s.cnt;
  const int64_t from = t0 > 0 ? t0 : 0;
  if (t1 <= from) return {0, 0};
  return {(int32_t)from * A.G.g, (int32_t)t1 * A.G.g};
}

// The exponent's part of a row: p = 2^(score * scale + shift). -infinity for a row that draws nothing, as for one with a score of infinity: every
// finite score's weight is zero then.
__device__ __forceinline__ float shift_of(const ChunkArgs& A, const Site& s, int32_t m) {
  if (m >= s.cnt * A.G.g) return -INFINITY;
  const int32_t t = m / A.G.g, j = m - t * A.G.g;
  const float x = A.lse[((int64_t)s.r * A.T + t) * A.G.Hq + s.h * A.G.g + j];
  return draws(x) ? -x * kLog2e : -INFINITY;
}

// Slots that nothing is added to.
__device__ __forceinline__ void copy_weights(const ChunkArgs& A, const Site& s) {
  const int64_t first = ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb + s.slot0;
  for (int32_t k = threadIdx.x; k < s.slots; k += blockDim.x) A.weight_out[first + k] = A.weight ? A.weight[first + k] : 0.f;
}

// ---- tensor cores: bf16 ------------------------------------------------------------------------------
//
// K of two tiles of up to 128 tokens stays in shared memory, the rows' queries come in tiles of up to 128 through a ring,
// each for both:
//   S = Q K^T   128 rows x 128 tokens, in two TMEM buffers of each tile
// Four warpgroups take half the tokens of a tile each. A thread has a row of S, whose log sum is a number of its own, and keeps a
// sum for each of its 64 tokens over all its rows; the sums of the warps' lanes are joined once, at the end. Per score that is
// an exponential, half a fused multiply-add and half an addition: exponentials and products both take 1024 cycles of
// two tiles. Four warps on a scheduler hide one another's waits. Slower: K Q^T, a token to a thread and its log sums from
// shared memory, 300 cycles and more a load beside the MMAs that read it; two warpgroups of 128 sums to a thread.
// Slots are listed as for the attention, so that few tiles need a mask.
constexpr int kTok = 128, kRing = 4, kWgs = 4, kThreads = kWgs * 128 + 128, kUpRegs = 104, kDownRegs = 64;  // 4 x 104 + 64 = 5 x 96

struct Bars {
  uint64_t k_full, full[kRing], empty[kRing], s_full[2][2], s_empty[2][2], drain;
  Listed listed;
  int32_t lo, hi, failed;
  uint32_t tmem;
};
__host__ __device__ constexpr size_t weigh_misc(int kb) { return sizeof(Bars) + ((size_t)kb * 2 + 15) / 16 * 16; }

struct WeighMaps {
  CUtensorMap tile, slot, q;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
weigh_mma_kernel(const ChunkArgs A, const __grid_constant__ WeighMaps M, const int32_t tiles, const int32_t rings, const int32_t q_tok, const int32_t pitch) {
  using L = Lines<D, kTok>;
  constexpr uint32_t kDesc = mma_desc_bf16(128, kTok, false);
  extern __shared__ __align__(1024) uint8_t smem_1024[];
  Bars& B = *reinterpret_cast<Bars*>(smem_1024);
  uint16_t* list_at = reinterpret_cast<uint16_t*>(&B + 1);
  const uint32_t begin = smem_u32(smem_1024), behind = begin + (uint32_t)weigh_misc(A.G.kb);
  uint8_t* ks = smem_1024 + ((behind + 1023) / 1024 * 1024 - begin);  // two tiles
  uint8_t* rs = ks + 2 * L::kBuf;                                      // [ring][chunks][128][line]
  // a kilobyte may be lost to where the block's memory begins
  const int32_t ring = min(rings, (int32_t)((begin + dynamic_smem() - smem_u32(rs)) / L::kBuf));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool is_copy = warp == 16, is_mma = warp == 17, is_soft = warp < 16, lists = warp < 8;
  const int32_t g = A.G.g, gr = q_tok * g, bs = A.G.bs, spt = kTok / pitch;
  if (is_copy) {
    if (lane < 3) tma_prefetch_map(&M.tile + lane);
    constexpr int kSE = offsetof(Bars, s_empty) / 8;
    for (int i = lane; i < (int)(offsetof(Bars, listed) / 8); i += 32) mbar_init(smem_u32(&B.k_full + i), i >= kSE && i < kSE + 4 ? 256 : 1);
    if (lane == 0) B.lo = INT32_MAX, B.hi = 0, B.failed = 0;
    fence_mbar_init();
    fence_proxy_async();
  }
  grid_wait();
  Span s;
  const int32_t ua = blockIdx.x / tiles, e0 = (blockIdx.x - ua * tiles) * 2 * spt;  // the CTA's entries begin at e0
  s.r = ua / A.G.Hkv;
  s.h = ua - s.r * A.G.Hkv;
  s.row0 = s.part = 0;
  s.parts = 1;
  const int64_t unit = (int64_t)ua * A.G.kb;
  Ids ids;
  if (lists) ids = load_ids(A, s, warp, 8);
  fill_span(A, INT32_MAX, s);
  uint32_t all[8] = {}, some[8] = {};
  auto copy_weights = [&] {  // of slots that no row sees
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u >= ids.per) break;
      const int32_t i = ids.first + u * 32 + lane;
      if (i < A.G.kb && !((all[u] | some[u]) >> lane & 1)) A.weight_out[unit + i] = A.weight ? A.weight[unit + i] : 0.f;
    }
  };
  if (s.rows <= 0) {
    grid_go();
    if (lists && e0 == 0) copy_weights();
    return;
  }
  if (lists) count_slots(A, s, ids, warp, B.listed, all, some);
  __syncthreads();
  if (lists) {
    place_slots(A, ids, warp, B.listed, all, some, list_at);
    if (e0 == 0) copy_weights();
  }
  __syncthreads();
  const List list = make_list(A, s, 8, B.listed, list_at);
  if (e0 >= list.n) {
    grid_go();
    return;
  }
  const int32_t ne = min(2 * spt, list.n - e0);
  // the rows that see any of them
  if (lists) {  // 256 threads: an entry each
    int32_t lo = INT32_MAX, hi = 0;
    if (tid < ne) {
      const int32_t e = e0 + tid;
      lo = 0, hi = s.rows;
      if (e >= list.whole) {
        const int32_t base = list.first(e);
        lo = max(0, base - s.len) * g;
        if (base >= A.sinks) {
          const int64_t last = (int64_t)base - s.len + bs - 1 + A.window;
          if (last < s.cnt) hi = max((int32_t)last, 0) * g;
        }
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0 && hi) atomicMin(&B.lo, lo), atomicMax(&B.hi, hi);
  } else if (is_mma) {
    tmem_alloc(smem_u32(&B.tmem), 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_go();  // the TMEM is allocated
  const uint32_t tmem = __shfl_sync(0xffffffffu, B.tmem, 0);
  const int32_t first = B.lo / gr, n = max(0, (B.hi + gr - 1) / gr - first);  // tiles of rows
  const int used = ne > spt ? 2 : 1;                                          // tiles
  auto warp_wait = [&](uint64_t& bar, int32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_timed(smem_u32(&bar), (uint32_t)parity)) != 0;
  };
  auto fail = [&] { *(volatile int32_t*)&B.failed = 1; };

  if (!is_soft) {
    registers_down<kDownRegs>();
    if (is_copy && n > 0) {
      const uint32_t k_bar = smem_u32(&B.k_full);
      if (lane == 0) mbar_expect_tx(k_bar, (uint32_t)(ne * bs * D * 2));
      __syncwarp();
      for (int t = 0; t < used; ++t) {
        const int32_t f0 = e0 + t * spt, nf = min(spt, list.n - f0), slot0 = list.slot(f0);
        const uint32_t to = smem_u32(ks) + t * L::kBuf;
        bool run = nf == spt && pitch == bs;
        for (int32_t e = lane; e < nf; e += 32) run = run && list.slot(f0 + e) == slot0 + e;
        if (__all_sync(0xffffffffu, run)) {
          if (lane < L::kChunks) tma_load_5d(to + lane * L::kChunk, &M.tile, k_bar, 0, lane, 0, 0, (int32_t)unit + slot0);
        } else {
          for (int32_t x = lane; x < nf * L::kChunks; x += 32) {
            const int32_t e = x / L::kChunks, c = x % L::kChunks;
            tma_load_5d(to + c * L::kChunk + e * pitch * L::kBytes, &M.slot, k_bar, 0, c, 0, 0, (int32_t)unit + list.slot(f0 + e));
          }
        }
      }
      int32_t issued = 0, b = 0, parity = 1;
      for (; issued < n; ++issued) {
        if (issued >= ring && !warp_wait(B.empty[b], parity)) {
          fail();
          break;
        }
        const uint32_t bar = smem_u32(&B.full[b]);
        if (lane == 0) mbar_expect_tx(bar, (uint32_t)(gr * D * 2));
        __syncwarp();
        if (lane < L::kChunks)
          tma_load_5d(smem_u32(rs) + b * L::kBuf + lane * L::kChunk, &M.q, bar, 0, lane, 0, s.h, s.r * A.T + (first + issued) * q_tok);
        if (++b == ring) b = 0, parity ^= 1;
      }
      // what is in flight lands before the shared memory is given up, whatever the others did (bounded)
      for (int32_t i = max(0, issued - ring); i < issued; ++i) mbar_wait_timed(smem_u32(&B.full[i % ring]), (i / ring) & 1);
      mbar_wait_timed(k_bar, 0);
    } else if (is_mma && n > 0) {
      if (elect_one()) {
        constexpr int kSteps = L::kElems / 16;
        constexpr uint32_t kHi = smem_desc_hi(L::kGroup, L::kSwizzle);
        const uint32_t kd = smem_desc_lo(smem_u32(ks), 16), qd = smem_desc_lo(smem_u32(rs), 16);
        bool ok = true;
        // barriers are asked ahead, behind MMAs that keep the tensor cores busy meanwhile
        auto ask = [&](uint64_t& bar, int32_t parity) { return mbar_test(smem_u32(&bar), (uint32_t)parity); };
        auto passed = [&](bool asked, uint64_t& bar, int32_t parity) {
          if (!asked) ok = ok && mbar_wait_timed(smem_u32(&bar), (uint32_t)parity);
          tc_fence_after();
        };
        passed(false, B.k_full, 0);
        bool q_there = false, s_there = false;
        int32_t b = 0, parity = 0;
        for (int32_t i = 0; i < n && ok; ++i) {
          const uint32_t q = qd + b * (L::kBuf >> 4);
          uint64_t& done = B.empty[b];
          passed(q_there, B.full[b], parity);
          if (++b == ring) b = 0, parity ^= 1;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (v == used) break;
            if (i > 1) passed(s_there, B.s_empty[v][i & 1], (i / 2 - 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              if (c == D / 32) {
                if (v + 1 < used) {
                  s_there = i > 1 && ask(B.s_empty[v + 1][i & 1], (i / 2 - 1) & 1);
                } else {
                  q_there = i + 1 < n && ask(B.full[b], parity);
                  s_there = i > 0 && ask(B.s_empty[0][(i + 1) & 1], ((i + 1) / 2 - 1) & 1);
                }
              }
              mma_ss1(tmem + v * 256 + (i & 1) * kTok, q + c / kSteps * (L::kChunk >> 4) + c % kSteps * 2,
                      kd + v * (L::kBuf >> 4) + c / kSteps * (L::kChunk >> 4) + c % kSteps * 2, kHi, kDesc, c > 0);
            }
            mma_commit1(smem_u32(&B.s_full[v][i & 1]));
          }
          if (ok) mma_commit1(smem_u32(&done));
        }
        if (!ok) fail();
        mma_commit1(smem_u32(&B.drain));
        mbar_wait_timed(smem_u32(&B.drain), 0);
      }
      __syncwarp();
    }
    __syncthreads();  // as the sums' warps below
    __syncthreads();
    if (is_mma) {
      tc_fence_after();
      tmem_free(tmem, 512);
    }
  } else {
    registers_up<kUpRegs>();
    const int w = warp >> 2, t = w >> 1, half = w & 1, row = tid & 127;
    const int32_t f0 = e0 + t * spt, nf = min(spt, list.n - f0);
    const bool masked = f0 + nf > list.whole;
    const float scale = kLog2e * rsqrtf((float)D);
    float2 acc[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) acc[c] = make_float2(0.f, 0.f);
    // the log sum of this thread's row of a tile, whose rows are q_tok tokens behind the last one's; of one that does not
    // count, as of one that sees nothing
    int32_t m = first * gr + row, p = s.len + m / g;  // of the row
    const float* lse_at = A.lse + row_place(A, s, m);
    const int32_t m_end = row < gr ? s.rows : 0;
    float lse = t < used && m < m_end ? *lse_at : -INFINITY;
    bool there = false;  // the next scores, asked for ahead
    for (int32_t i = 0; i < n && t < used; ++i, p += q_tok) {
      m += gr;
      lse_at += q_tok * A.G.Hq;
      const float next = i + 1 < n && m < m_end ? *lse_at : -INFINITY;  // on its way for a tile's time
      uint64_t vis = draws(lse) ? ~0ull : 0;
      if (masked && vis) {
        vis = 0;
#pragma unroll 1
        for (int32_t k = 0; k < nf; ++k) {
          const int32_t at = k * pitch - half * 64;
          if (at >= 64 || at + bs <= 0) continue;
          const uint64_t bits = list.seen(f0 + k, p, A.window, A.sinks);
          vis |= at >= 0 ? bits << at : bits >> -at;
        }
      }
      if (!__all_sync(0xffffffffu, there) && !warp_wait(B.s_full[t][i & 1], (i >> 1) & 1)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t at = tmem + t * 256 + ((uint32_t)(warp & 3) << 21) + (i & 1) * kTok + half * 64;
      const float2 scale2 = make_float2(scale, scale), shift2 = make_float2(-lse * kLog2e, -lse * kLog2e);
      // twice, with the loads: one loop for both takes the mask's tests for every score, three instructions to two of the sums
      auto add = [&](auto with_mask) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t x[16];
          tmem_ld16(x, at + q * 16);
          tmem_wait_ld(x);
          if (q == 3) {
            tc_fence_before();
            mbar_arrive(smem_u32(&B.s_empty[t][i & 1]));
            there = i + 1 < n && mbar_test(smem_u32(&B.s_full[t][(i + 1) & 1]), ((i + 1) >> 1) & 1);
          }
          const uint32_t bits = (uint32_t)(vis >> 16 * q);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 p = fma2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), scale2, shift2);
            float2 e = make_float2(ex2(p.x), ex2(p.y));
            if (with_mask) e = make_float2(bits >> (2 * c) & 1 ? e.x : 0.f, bits >> (2 * c + 1) & 1 ? e.y : 0.f);
            acc[q * 8 + c] = add2(acc[q * 8 + c], e);
          }
        }
      };
      if (__any_sync(0xffffffffu, masked || !vis))
        add(std::true_type());
      else
        add(std::false_type());
      lse = next;
    }
    // over the lanes: each step hands half of a lane's tokens to its partner; tokens 2 lane and 2 lane + 1 are left
    float v[64];
#pragma unroll
    for (int c = 0; c < 32; ++c) v[2 * c] = acc[c].x, v[2 * c + 1] = acc[c].y;
#pragma unroll
    for (int step = 32; step >= 2; step /= 2) {
      const bool up = lane & (step / 2);
#pragma unroll
      for (int c = 0; c < step; ++c) {
        const float keep = up ? v[c + step] : v[c], give = up ? v[c] : v[c + step];
        v[c] = keep + __shfl_xor_sync(0xffffffffu, give, step / 2);
      }
    }
    __syncthreads();  // nothing reads or fills the ring any more
    float* part = reinterpret_cast<float*>(rs);  // [tiles][warps of a quarter][128]
    *reinterpret_cast<float2*>(part + (t * 4 + (warp & 3)) * 128 + half * 64 + lane * 2) = make_float2(v[0], v[1]);
    asm volatile("bar.sync %0, 256;" ::"r"(t + 1) : "memory");
    const bool failed = *(volatile int32_t*)&B.failed != 0;
    for (int32_t k = tid & 255; k < nf; k += 256) {
      const int64_t at = unit + list.slot(f0 + k);
      const float* x = part + t * 512 + k * pitch;
      float sum = 0.f;
      for (int32_t j = 0; j < bs && !failed; ++j) sum += (x[j] + x[j + 128]) + (x[j + 256] + x[j + 384]);
      A.weight_out[at] = (A.weight ? A.weight[at] : 0.f) + sum;
    }
    tc_fence_before();
    __syncthreads();
  }
}

// ---- binary32 ------------------------------------------------------------------------------------------
//
// Products of three parts (mma_f32), K of 64 tokens as the rows, queries in tiles of 32 as the columns; a score that is not
// finite (an operand's parts may not add up to it) is taken again by plain products. A warp has 16 tokens.
constexpr int kF32Tok = 64, kF32Rows = 32, kF32Threads = 128;
__host__ __device__ constexpr int f32_pitch(int d) { return d + 4; }
__host__ __device__ constexpr size_t f32_smem(int d) { return (size_t)(kF32Tok + kF32Rows) * f32_pitch(d) * 4 + (kF32Rows + kF32Tok) * 4 + 16; }

template <int DV>
__global__ void __launch_bounds__(kF32Threads) weigh_f32_kernel(const ChunkArgs A, const int32_t tiles, const int32_t q_tok) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int d = DV * 32, pitch = f32_pitch(d), kPieces = d / 4, NT = kF32Rows / 8;
  float* ks = reinterpret_cast<float*>(smem);  // [64][pitch]
  float* qs = ks + kF32Tok * pitch;            // [32][pitch]
  float* shift = qs + kF32Rows * pitch;        // [32]
  float* part = shift + kF32Rows;              // [64]
  int32_t* range = reinterpret_cast<int32_t*>(part + kF32Tok);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, ti = lane & 3;
  const int32_t g = A.G.g, gr = q_tok * g, bs = A.G.bs, spt = kF32Tok / bs;
  if (tid == 0) range[0] = INT32_MAX, range[1] = 0;
  grid_wait();
  grid_go();
  const Site s = make_site(A, spt, tiles);
  const int64_t unit = ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb;
  auto rows_at = [&](int32_t j) {
    const int32_t k = j / bs;
    return k < s.slots ? rows_of(A, s, A.slot_block[unit + s.slot0 + k], j - k * bs) : Rows{0, 0};
  };
  const Rows mine[2] = {rows_at(warp * 16 + gi), rows_at(warp * 16 + gi + 8)};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t lo = __reduce_min_sync(0xffffffffu, mine[i].lo < mine[i].hi ? mine[i].lo : INT32_MAX), hi = __reduce_max_sync(0xffffffffu, mine[i].hi);
    if (lane == 0 && hi) atomicMin(&range[0], lo), atomicMax(&range[1], hi);
  }
  __syncthreads();
  if (range[1] == 0) {
    copy_weights(A, s);
    return;
  }
  const int32_t first = range[0] / gr, end = (range[1] + gr - 1) / gr;
  for (int32_t i = tid; i < kF32Tok * kPieces; i += kF32Threads) {
    const int32_t j = i / kPieces, c = i % kPieces, k = j / bs;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < s.slots) x = *reinterpret_cast<const float4*>(A.pool + (unit + s.slot0 + k) * A.G.block_bytes + ((int64_t)(j - k * bs) * d + c * 4) * 4);
    *reinterpret_cast<float4*>(ks + j * pitch + c * 4) = x;
  }
  const float scale = kLog2e / sqrtf((float)d);
  float total[2] = {0.f, 0.f};
  // a tile of queries comes into registers while the one before is at its products
  constexpr int kEach = kF32Rows * kPieces / kF32Threads;
  float4 rows[kEach];
  float row_shift = 0.f;
  auto fetch = [&](int32_t i) {
    const int32_t m0 = i * gr;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int32_t x = tid + u * kF32Threads, row = x / kPieces, c = x % kPieces, m = m0 + row, t = m / g;
      rows[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < end && row < gr && t < s.cnt)
        rows[u] = *reinterpret_cast<const float4*>((const float*)A.q + ((((int64_t)s.r * A.T + t) * A.G.Hq + s.h * g + m - t * g) * d + c * 4));
    }
    if (tid < kF32Rows) row_shift = i < end && tid < gr ? shift_of(A, s, m0 + tid) : -INFINITY;
  };
  fetch(first);
  for (int32_t i = first; i < end; ++i) {
    const int32_t m0 = i * gr;
    __syncthreads();  // the tile before has been read
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int32_t x = tid + u * kF32Threads;
      *reinterpret_cast<float4*>(qs + x / kPieces * pitch + x % kPieces * 4) = rows[u];
    }
    if (tid < kF32Rows) shift[tid] = row_shift;
    __syncthreads();
    fetch(i + 1);
    float sc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
    const float* ka = ks + (warp * 16 + gi) * pitch + ti;
    const float* qr = qs + gi * pitch + ti;
#pragma unroll 4
    for (int k = 0; k < d; k += 8) {
      const Parts a[4] = {parts_of(ka[k]), parts_of(ka[k + 8 * pitch]), parts_of(ka[k + 4]), parts_of(ka[k + 8 * pitch + 4])};
      Parts b[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n][0] = parts_of(qr[n * 8 * pitch + k]), b[n][1] = parts_of(qr[n * 8 * pitch + k + 4]);
      mma_f32<NT>(sc, a, b);
    }
    // tokens gi (sc[.][0], sc[.][1]) and gi + 8; rows 8 n + 2 ti and the next
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 8 * n + 2 * ti + (e & 1);
        const Rows& v = mine[e >> 1];
        if (m0 + row < v.lo || m0 + row >= v.hi || row >= gr) continue;
        float x = sc[n][e];
        if (!is_finite(x)) {
          const float *y = ks + (warp * 16 + gi + 8 * (e >> 1)) * pitch, *z = qs + row * pitch;
          x = 0.f;
#pragma unroll 1
          for (int k = 0; k < d; ++k) x = fmaf(y[k], z[k], x);
        }
        sum[e >> 1] += ex2(fmaf(x, scale, shift[row]));
      }
    total[0] += sum[0];
    total[1] += sum[1];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    total[i] += __shfl_xor_sync(0xffffffffu, total[i], 1);
    total[i] += __shfl_xor_sync(0xffffffffu, total[i], 2);
    if (ti == 0) part[warp * 16 + gi + 8 * i] = total[i];
  }
  __syncthreads();
  for (int32_t e = tid; e < s.slots; e += kF32Threads) {
    const int64_t at = unit + s.slot0 + e;
    float sum = 0.f;
    for (int32_t i = e * bs; i < e * bs + bs; ++i) sum += part[i];
    A.weight_out[at] = (A.weight ? A.weight[at] : 0.f) + sum;
  }
}

// ---- launches ----------------------------------------------------------------------------------------------

template <typename... P, typename... Q>
cudaError_t launch_plain(void (*kernel)(P...), int64_t ctas, int threads, size_t smem, cudaStream_t s, Q&&... args) {
  return launch_cluster(kernel, ctas, Shape{1, (int32_t)ctas, 1}, threads, smem, s, std::forward<Q>(args)...);
}

template <int DV>
cudaError_t run_f32(const ChunkArgs& A, cudaStream_t s) {
  const int32_t spt = kF32Tok / A.G.bs, tiles = (A.G.kb + spt - 1) / spt;
  return launch_plain(weigh_f32_kernel<DV>, (int64_t)A.G.R * A.G.Hkv * tiles, kF32Threads, f32_smem(DV * 32), s, A, tiles, kF32Rows / A.G.g);
}

template <int D>
cudaError_t run_mma(const ChunkArgs& A, cudaStream_t s) {
  using L = Lines<D, kTok>;
  const int32_t pitch = A.G.bs * L::kBytes % 128 ? A.G.bs + 1 : A.G.bs, spt = kTok / pitch, tiles = (A.G.kb + 2 * spt - 1) / (2 * spt);
  const int32_t q_tok = A.T < 128 / A.G.g ? A.T : 128 / A.G.g;
  // one CTA to an SM, by its TMEM: never so small that another kernel's that takes TMEM finds a place beside it
  const size_t rest = (weigh_misc(A.G.kb) + 1023) / 1024 * 1024 + 2 * L::kBuf, least = 2 * (233472 / 3);
  int32_t ring = (int32_t)((kMaxSmem - rest) / L::kBuf);
  if (ring > kRing) ring = kRing;
  size_t smem = rest + (size_t)ring * L::kBuf + 1024;
  if (smem > kMaxSmem) smem = kMaxSmem;
  if (smem < least) smem = least;
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  WeighMaps m;
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
  if (!encode(&m.tile, A.pool, {bs, 2, slots}, {token, half, 2 * half}, {(cuuint32_t)bs, 1, (cuuint32_t)spt}) ||
      !encode(&m.slot, A.pool, {bs, 2, slots}, {token, half, 2 * half}, {(cuuint32_t)bs, 1, 1}) ||
      !encode(&m.q, A.q, {g, hkv, all}, {token, token * g, token * g * hkv}, {(cuuint32_t)g, 1, (cuuint32_t)q_tok}))
    return cudaErrorInvalidValue;
  return launch_plain(weigh_mma_kernel<D>, (int64_t)A.G.R * A.G.Hkv * tiles, kThreads, smem, s, A, m, tiles, ring, q_tok, pitch);
}

}  // namespace

cudaError_t launch_weigh_chunk(const ChunkArgs& A, cudaStream_t s) {
  const int32_t v = A.G.d / 32;
  if (A.G.dtype == OKV_F32) {
    switch (v) {
      case 1: return run_f32<1>(A, s);
      case 2: return run_f32<2>(A, s);
      case 3: return run_f32<3>(A, s);
      case 4: return run_f32<4>(A, s);
      case 5: return run_f32<5>(A, s);
      case 6: return run_f32<6>(A, s);
      case 7: return run_f32<7>(A, s);
      default: return run_f32<8>(A, s);
    }
  }
  switch (v) {
    case 1: return run_mma<32>(A, s);
    case 2: return run_mma<64>(A, s);
    case 3: return run_mma<96>(A, s);
    case 4: return run_mma<128>(A, s);
    case 5: return run_mma<160>(A, s);
    case 6: return run_mma<192>(A, s);
    case 7: return run_mma<224>(A, s);
    default: return run_mma<256>(A, s);
  }
}

}  // namespace okv
