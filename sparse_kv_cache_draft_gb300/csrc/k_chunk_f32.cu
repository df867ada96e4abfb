// Attention of a chunk of new tokens over a paged pool, binary32: what k_chunk.cu says of rows, lists and clusters holds here.
//
// Products of three parts on the tensor cores (mma_f32), as for drafted trees: 128 threads, 16 RG rows x 64 tokens; a warp
// takes 16 rows and 64 / TH of the tokens with a maximum, sum and output of its own, merged at the end. The parts of an operand
// that is not finite, or next to the largest number, do not add up to it: a score is then NaN and an output NaN or
// infinite, so a CTA that ends with a sum or an output that is not finite takes its tiles again by plain products.
#include "chunk.cuh"

namespace okv {
namespace {

constexpr int kF32Tile = 64, kF32Threads = 128;

__host__ __device__ constexpr int f32_pitch(int d) { return d + 4; }  // fragment reads free of bank conflicts
__host__ __device__ constexpr size_t f32_smem(int d, int rg, int stages, int kb) {
  const int th = 4 / rg;
  return (size_t)(16 * rg + 2 * stages * kF32Tile) * f32_pitch(d) * 4 + (size_t)(th + 1) * 16 * rg * 8 + 48 + sizeof(Listed) + ((size_t)kb * 2 + 15) / 16 * 16;
}
// CTAs of an SM, by registers, or one with two stages of tiles
__host__ __device__ constexpr int f32_ctas(int dv, int rg, int stages) { return stages == 2 ? 1 : dv <= 4 && rg < 4 ? 3 : dv <= 4 ? 2 : 1; }

// Where CTAs are few a tile's keys and values come while the one before it is at work (ST = 2); otherwise the CTAs of an SM hide
// one another's waits, with room for more of them.
template <int DV, int RG, int ST>
__global__ void __launch_bounds__(kF32Threads, f32_ctas(DV, RG, ST)) chunk_f32_kernel(const __grid_constant__ ChunkArgs A, const Shape shape, const int32_t q_tok) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int d = DV * 32, pitch = f32_pitch(d), kRows = 16 * RG, TH = 4 / RG, kTok = kF32Tile / TH, NT = kTok / 8;
  float* qs = reinterpret_cast<float*>(smem);      // [rows][pitch]
  float* ks0 = qs + kRows * pitch;                 // [ST][64][pitch]
  float* vs0 = ks0 + ST * kF32Tile * pitch;        // [ST][64][pitch]
  float* ms = vs0 + ST * kF32Tile * pitch;         // [rows], then [TH][rows] of the warps
  float* ls = ms + (TH + 1) * kRows;               // the same
  uint64_t* bars = reinterpret_cast<uint64_t*>(ls + (TH + 1) * kRows);  // keys, values (of a stage), queries there
  uint64_t* q_bar = bars + 2 * ST;
  int32_t* bad = reinterpret_cast<int32_t*>(q_bar + 1);
  Listed& listed = *reinterpret_cast<Listed*>(bars + 6);
  uint16_t* list_at = reinterpret_cast<uint16_t*>(&listed + 1);

  if (threadIdx.x == 0) {
    *bad = 0;
    for (int i = 0; i < 2 * ST; ++i) mbar_init(smem_u32(bars + i), kF32Tile);
    mbar_init(smem_u32(q_bar), kRows);
    fence_mbar_init();
    fence_proxy_async();
  }
  __syncthreads();
  grid_wait();
  grid_go();
  const int32_t g = A.G.g;
  Span s = make_span(A, shape, q_tok * g);
  const Ids ids = load_ids(A, s, threadIdx.x >> 5, 4);
  fill_span(A, q_tok * g, s);
  if (s.rows <= 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, ti = lane & 3;
  const int rg = warp % RG, th = warp / RG, tok0 = th * kTok;
  const int32_t bs = A.G.bs, spt = kF32Tile / bs, tt = spt * bs;
  const int64_t unit = ((int64_t)s.r * A.G.Hkv + s.h) * A.G.kb;
  constexpr int kPieces = d / 4, kEach = kF32Tile * kPieces / kF32Threads;  // 16-byte pieces of a token, of a thread's share of a tile
  // Rows are copied whole, each by a thread that counts it at the barrier of its tile.
  auto copy_row = [&](uint32_t bar, float* to, const float* from) {
    mbar_expect_tx(bar, d * 4);
    bulk_load(smem_u32(to), from, d * 4, bar);
  };
  if (tid < kRows) {  // rows past the group's are never read out
    if (tid < s.rows)
      copy_row(smem_u32(q_bar), qs + tid * pitch, (const float*)A.q + row_place(A, s, s.row0 + tid) * d);
    else
      mbar_arrive(smem_u32(q_bar));
  }
  uint32_t whole_of[8], some_of[8];
  count_slots(A, s, ids, warp, listed, whole_of, some_of);
  __syncthreads();
  place_slots(A, ids, warp, listed, whole_of, some_of, list_at);
  __syncthreads();
  const List list = make_list(A, s, 4, listed, list_at);
  const int32_t mine = ((list.n + spt - 1) / spt - s.part + s.parts - 1) / s.parts;  // this CTA's tiles
  const float scale = kLog2e / sqrtf((float)d);
  const uint32_t per_bs = (65536 + bs - 1) / bs;  // j * per_bs >> 16 is j / bs for j < 64
  auto first_of = [&](int32_t it) { return (s.part + it * s.parts) * spt; };
  bool failed = false, again = false;
  auto use = [&](int32_t it) { return again ? mine + it : it; };
  auto stage = [&](int32_t it) { return ST == 2 ? use(it) & 1 : 0; };
  auto there = [&](int32_t it, int which) {
    return mbar_wait_timed(smem_u32(bars + 2 * stage(it) + which), (uint32_t)(ST == 2 ? use(it) >> 1 : use(it)) & 1);
  };
  // Tile it's keys (which = 0) or values into shared memory, by 64 threads, a token each. A value that no row may see
  // is zero, as its weight of zero needs; a key may be anything.
  auto load = [&](int32_t it, int which) {
    if (it >= mine) return;
    const int32_t j = tid & 63, in = j * per_bs >> 16, off = j - in * bs, e = first_of(it) + in;
    const float* from = nullptr;
    if (j < tt && e < list.n) {
      const int32_t slot = list.slot(e);
      if (e < list.whole || list.first(e) <= s.p_hi - off)
        from = reinterpret_cast<const float*>(A.pool + (unit + slot) * A.G.block_bytes) + (int64_t)(which * bs + off) * d;
    }
    const uint32_t bar = smem_u32(bars + 2 * stage(it) + which);
    float* to = (which ? vs0 : ks0) + (stage(it) * kF32Tile + j) * pitch;
    if (from) {
      copy_row(bar, to, from);
    } else {
      if (which)
        for (int c = 0; c < d; c += 4) *reinterpret_cast<float4*>(to + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      mbar_arrive(bar);
    }
  };
  load(0, tid >> 6);

  bool real[2];
  int32_t pos[2];  // of rows gi and gi + 8 of the warp's 16
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t row = rg * 16 + gi + 8 * i;
    real[i] = row < s.rows;
    pos[i] = s.len + (s.row0 + row) / g;
  }
  float o[d / 8][4], m[2], l[2];
  bool ok = mbar_wait_timed(smem_u32(q_bar), 0);
  for (;;) {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < d / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    for (int32_t it = 0; it < mine && !failed; ++it) {
      const int32_t e0 = first_of(it);
      const bool part_seen = e0 + spt > list.whole;
      const float* ks = ks0 + stage(it) * kF32Tile * pitch;
      float* vs = vs0 + stage(it) * kF32Tile * pitch;
      if (ST == 2) {
        fence_proxy_async();  // zeros were written among the values of the tile before the last
        load(it + 1, tid >> 6);
      }
      uint64_t vis[2] = {first_bits(real[0] ? tt : 0), first_bits(real[1] ? tt : 0)};
      if (part_seen) {
        vis[0] = vis[1] = 0;
        const int32_t ne = min(spt, list.n - e0);
#pragma unroll 1
        for (int32_t k = 0; k < ne; ++k) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (real[i]) vis[i] |= list.seen(e0 + k, pos[i], A.window, A.sinks) << k * bs;
        }
      }
      ok = there(it, 0) && ok;
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
      const float* qa = qs + (rg * 16 + gi) * pitch + ti;
      const float* kr = ks + (tok0 + gi) * pitch + ti;
#pragma unroll(NT > 4 ? 2 : 4)
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
        const float mn = larger_max(m[i], mx), ref = mn == -INFINITY ? 0.f : mn, f = ex2(m[i] - ref);
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
      if (ST == 1) {
        __syncthreads();
        if (tid < 64) load(it + 1, 0);  // the keys have been read
      }
      ok = there(it, 1) && ok;
      if (part_seen) {
        // values that are not finite are zero in the products
#pragma unroll 1
        for (int u = 0; u < kEach; ++u) {
          const int i = tid + u * kF32Threads, j = i / kPieces, c = i % kPieces;
          float4* at = reinterpret_cast<float4*>(vs + j * pitch + c * 4);
          float4 y = *at;
          if (is_finite(y.x) && is_finite(y.y) && is_finite(y.z) && is_finite(y.w)) continue;
          *(volatile int32_t*)bad = 1;
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
      if (ST == 1 && tid >= 64 && !failed) {  // the values have been read
        fence_proxy_async();                  // zeros were written among them
        load(it + 1, 1);
      }
      if (failed && it + 1 < mine) {  // copies in flight land (bounded)
        there(it + 1, 0);
        if (ST == 2) there(it + 1, 1);
      }
    }
    bool odd = real[0] && !is_finite(l[0]) || real[1] && !is_finite(l[1]);
#pragma unroll
    for (int n = 0; n < d / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) odd |= real[e >> 1] && !is_finite(o[n][e]);
    if (again || failed || !__syncthreads_or(odd)) break;
    fence_proxy_async();
    again = true;
    load(0, tid >> 6);
  }
  float* ks = ks0;
  if (failed || !ok) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const RowSums end = sums_at_end(true, m[i], l[i]);
      m[i] = end.m, l[i] = end.l;
    }
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
    if (*bad && sum != 0.f) {
      const float4 y = not_finite_of<float>(A, unit, list.at, list.base, list.whole, list.n, s.part, s.parts, spt, s.len + (s.row0 + row) / g, c * 4);
      x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    if (s.parts > 1) {
      *reinterpret_cast<float4*>(ks + row * d + c * 4) = x;  // read above by this thread alone
      if (c == 0) {
        ms[row] = M;
        ls[row] = sum;
      }
      continue;
    }
    const float inv = 1.f / sum;
    x = sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    const int64_t at = row_place(A, s, s.row0 + row);
    store4((float*)A.out + at * d + c * 4, x);
    if (c == 0 && A.lse) A.lse[at] = lse_of(M, sum);
  }
  if (s.parts > 1) merge_chunk<float>(A, s, Partial{smem_u32(ks), smem_u32(ms), smem_u32(ls)}, 0, kF32Threads, [] {});
}

// ---- launches ----------------------------------------------------------------------------------------------

constexpr Costs kF32Costs{2.8, 0.5, 1.3};  // those of the drafted trees, where a CTA has one stage of tiles

template <int DV, int RG, int ST>
cudaError_t run_f32(const ChunkArgs& A, cudaStream_t s) {
  const int32_t q_tok = 16 * RG / A.G.g, groups = (A.T + q_tok - 1) / q_tok;
  const size_t smem = f32_smem(DV * 32, RG, ST, A.G.kb);
  int32_t per_sm = (int32_t)(228 * 1024 / (smem + 1024));
  if (per_sm > f32_ctas(DV, RG, ST)) per_sm = f32_ctas(DV, RG, ST);
  if (per_sm < 1) per_sm = 1;
  const int64_t items = (int64_t)A.G.R * A.G.Hkv * groups;
  const Shape shape = pick_shape(items, groups, per_sm, likely_tiles(A, kF32Tile / A.G.bs, q_tok), kF32Costs, cluster_room(kF32Threads, per_sm));
  return launch_cluster(chunk_f32_kernel<DV, RG, ST>, items, shape, kF32Threads, smem, s, A, shape, q_tok);
}

// Rows of a CTA: 64 share a tile's keys and values four ways, but where even the largest clusters would leave SMs empty fewer
// rows end sooner (1 request x 40 tokens, 8 / 2 heads of 128 dims, 3000 tokens of context: 50 us by 64, 42 by 32, 30 by 16; 4 x 512
// tokens: 509, 632, 703). Two stages of tiles where an SM has one CTA anyway (1 token, 16 / 8 heads, 12K of context: 53 us against 81;
// 40 tokens as above, with more CTAs than SMs, 30.6 against 29.7).
template <int DV>
cudaError_t run_f32_rows(const ChunkArgs& A, cudaStream_t s) {
  const int32_t rows = A.T * A.G.g, sms = sm_count();
  auto ctas = [&](int32_t of) {  // at most
    const int32_t q_tok = of / A.G.g;
    return (int64_t)A.G.R * A.G.Hkv * ((A.T + q_tok - 1) / q_tok) * kMaxSplit;
  };
  if (rows <= 16 || ctas(32) < sms) {
    if constexpr (DV <= 6) {  // by shared memory
      if (ctas(16) <= sms) return run_f32<DV, 1, 2>(A, s);
    }
    return run_f32<DV, 1, 1>(A, s);
  }
  if (rows <= 32 || ctas(64) < sms) return run_f32<DV, 2, 1>(A, s);
  return run_f32<DV, 4, 1>(A, s);
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkArgs& A, cudaStream_t s) {
  switch (A.G.d / 32) {
    case 1: return run_f32_rows<1>(A, s);
    case 2: return run_f32_rows<2>(A, s);
    case 3: return run_f32_rows<3>(A, s);
    case 4: return run_f32_rows<4>(A, s);
    case 5: return run_f32_rows<5>(A, s);
    case 6: return run_f32_rows<6>(A, s);
    case 7: return run_f32_rows<7>(A, s);
    default: return run_f32_rows<8>(A, s);
  }
}

}  // namespace okv
