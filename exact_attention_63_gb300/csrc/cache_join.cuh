// The second kernel of attention over a paged cache: joins what the first one's CTAs left
// of tiles that more than one of them worked on.  `Plan::of(p, s)` gives sequence s's key
// blocks as the first kernel counts them.
#pragma once

#include <type_traits>

#include "cache_plan.cuh"

namespace attn {
namespace {

// Joins the parts of the tiles that were split.  With the parts' maxima m_i and
// sums l_i:  m = max m_i,  O = Σ 2^(m_i − m) O_i / Σ 2^(m_i − m) l_i.
// WAY = kJoinFew: a block takes one row, its eight warps deal out the parts (few rows;
// one long sequence leaves a part on every CTA).  kJoinRows: a block takes 32 rows, a
// warp four at once.  kJoinWide: parts that lie chunk by chunk; a block takes 32 rows,
// a lane a row, a warp a quarter of its values.  kJoinEight: a block takes 8 rows, a warp
// one with all of its parts (tiles of 8 or 16 rows, of which half and more may be empty).
enum { kJoinFew, kJoinRows, kJoinWide, kJoinEight };
constexpr int kEightRows = 16;

// The last s with tab[s] <= u of s in [0, n), tab[0] <= u: the warp tries 32 places at a time.
__device__ __forceinline__ int find_seq_warp(const int* tab, int n, int u, int lane) {
  int lo = 0, hi = n;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + step * lane;
    const uint32_t below = __ballot_sync(0xffffffffu, at < hi && tab[at] <= u);
    lo += step * (31 - __clz(below));
    hi = min(hi, lo + step);
  }
  return lo;
}

template <int D, int WAY, class Plan>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttnParams p, int grid, int mt_max, int ends) {
  constexpr int kPer = D / 32, SPLIT = WAY == kJoinEight ? 1 : 8;
  __shared__ float s_acc[WAY == kJoinFew ? SPLIT : 1][D];
  __shared__ float2 s_ml[SPLIT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kRows = WAY == kJoinFew ? 1 : WAY == kJoinEight ? 8 : 32;  // of a block
  const unsigned int chunks = (p.rows + kRows - 1) / kRows;
  const int hg = heads_of<Plan>(p);
  unsigned int x = blockIdx.x;
  const int row0 = static_cast<int>(x % chunks) * kRows;
  x /= chunks;
  int m, h, s, ua, units;
  KeyPlan k;
  auto cta_of = [&](int u) { return static_cast<int>(((u + 1ll) * grid - 1) / units); };
  if (Plan::kEight && ends) {
    // The block's tile is the one that the end of a CTA's range divides.
    const int c = static_cast<int>(x / hg) + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    units = p.ws_table[p.c.n_seq];
    grid = min(grid, units);
    if (c >= grid) return;
    const int u = range_start(units, c, grid);
    s = find_seq_warp(p.ws_table, p.c.n_seq, u, lane);
    k = Plan::of(p, s);
    const int rem = u - p.ws_table[s], hm = rem / (k.db + 1), mt = row_tiles(p, k.n);
    ua = u - (rem - hm * (k.db + 1));
    if (ua == u || cta_of(ua) != c - 1) return;  // no tile, or an earlier end's
    m = hm % mt;
    h = hm / mt * hg + static_cast<int>(x % hg);
  } else {
    m = static_cast<int>(x % mt_max);
    x /= mt_max;
    h = static_cast<int>(x % p.c.hkv);
    s = static_cast<int>(x / p.c.hkv);
    k = Plan::of(p, s);
    // The attention kernel's results, complete and visible.  Every block waits, so
    // that this kernel never ends before that one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    units = p.ws_table[p.c.n_seq];
    grid = min(grid, units);
    ua = p.ws_table[s] + (h / hg * row_tiles(p, k.n) + m) * (k.db + 1);
  }
  const int grp = p.c.group, first_row = m * p.rows, n_rows = min(k.n * grp - first_row, p.rows), nb = k.db + 1;
  if (row0 >= n_rows) return;
  const int c0 = cta_of(ua), c1 = cta_of(ua + nb - 1);
  if (c0 == c1) return;  // one CTA did it all and has written the rows
  // Every CTA's part but the first's is the first of its range.
  const int slot0 = 2 * c0 + (range_start(units, c0, grid) >= ua ? 0 : 1);
  const int in_run = h % hg;
  auto slot_of = [&](int c) { return static_cast<long long>(c == c0 ? slot0 : 2 * c) * hg + in_run; };
  auto part_of = [&](int c, int r) { return slot_of(c) * p.rows + r; };

  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  auto load = [&](int c, int r) { return *reinterpret_cast<const Vec*>(p.ws_o + part_of(c, r) * D + lane * kPer); };
  auto add = [&](float(&acc)[kPer], float w, const Vec& y) {
    const float* v = reinterpret_cast<const float*>(&y);
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] += w * v[i];
  };
  // Row r's output from the joined sums; one lane writes its LSE.
  auto finish = [&](int r, float mx, float sum, const float(&acc)[kPer], bool lse) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int hq = h * grp + (first_row + r) % grp;
    const long long token = k.q0 + (first_row + r) / grp;
    uint16_t* const dst = p.o + (token * p.c.hkv * grp + hq) * D + lane * kPer;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lse)
      p.lse[static_cast<long long>(hq) * p.c.total + token] =
          sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.69314718055994531f;
  };

  if constexpr (WAY == kJoinWide) {
    constexpr int kChunks = D / 16;  // of four values, of this warp
    const int r = min(row0 + lane, n_rows - 1), first = warp * kChunks;
    float mx = -INFINITY, sum = 0.f, acc2[kChunks][4] = {};
    for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, p.ws_ml[part_of(c, r)].x);
#pragma unroll 2
    for (int c = c0; c <= c1; ++c) {
      const float2 ml = p.ws_ml[part_of(c, r)];
      const float w = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - mx);
      sum += w * ml.y;
      const float4* src = reinterpret_cast<const float4*>(p.ws_o) +
                          (slot_of(c) * (D / 4) + first) * p.rows + r;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const float4 y = src[static_cast<long long>(i) * p.rows];
        acc2[i][0] += w * y.x;
        acc2[i][1] += w * y.y;
        acc2[i][2] += w * y.z;
        acc2[i][3] += w * y.w;
      }
    }
    if (row0 + lane >= n_rows) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int hq = h * grp + (first_row + r) % grp;
    const long long token = k.q0 + (first_row + r) / grp;
    uint4* const dst = reinterpret_cast<uint4*>(p.o + (token * p.c.hkv * grp + hq) * D + first * 4);
#pragma unroll
    for (int i = 0; i < kChunks; i += 2)
      dst[i / 2] = make_uint4(pack_bf16x2(acc2[i][0] * inv, acc2[i][1] * inv), pack_bf16x2(acc2[i][2] * inv, acc2[i][3] * inv),
                              pack_bf16x2(acc2[i + 1][0] * inv, acc2[i + 1][1] * inv),
                              pack_bf16x2(acc2[i + 1][2] * inv, acc2[i + 1][3] * inv));
    if (warp == 0)
      p.lse[static_cast<long long>(hq) * p.c.total + token] =
          sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.69314718055994531f;
  } else if constexpr (WAY == kJoinRows) {
    // Eight lanes a row look at its parts' maxima and sums.
    const int r0 = row0 + 4 * warp, mine = min(r0 + (lane >> 3), n_rows - 1);
    if (r0 >= n_rows) return;
    float mx = -INFINITY, sum = 0.f, acc[4][kPer] = {};
    for (int c = c0 + (lane & 7); c <= c1; c += 8) mx = fmaxf(mx, p.ws_ml[part_of(c, mine)].x);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    for (int cb = c0; cb <= c1; cb += 8) {
      const int c = cb + (lane & 7);
      float w = 0.f;
      if (c <= c1) {
        const float2 ml = p.ws_ml[part_of(c, mine)];
        w = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - mx);
        sum += w * ml.y;
      }
      const int n = min(8, c1 - cb + 1);
      for (int i = 0; i < n; i += 4) {  // four parts of four rows in flight; behind the last, weight 0
        Vec y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = load(min(cb + i + (e >> 2), c1), min(r0 + (e & 3), n_rows - 1));
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float we = __shfl_sync(0xffffffffu, w, 8 * (e & 3) + i + (e >> 2));
          if (we != 0.f) add(acc[e & 3], we, y[e]);
        }
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float m_j = __shfl_sync(0xffffffffu, mx, 8 * j), s_j = __shfl_sync(0xffffffffu, sum, 8 * j);
      if (r0 + j < n_rows) finish(r0 + j, m_j, s_j, acc[j], lane == 8 * j);
    }
  } else {
    const int r = WAY == kJoinEight ? row0 + warp : row0, mine = WAY == kJoinEight ? 0 : warp;
    if (r >= n_rows) return;
    float mx = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int c = c0 + mine + lane * SPLIT; c <= c1; c += 32 * SPLIT) mx = fmaxf(mx, p.ws_ml[part_of(c, r)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    for (int cb = c0 + mine; cb <= c1; cb += 32 * SPLIT) {
      const int c = cb + lane * SPLIT;
      float w = 0.f;
      if (c <= c1) {
        const float2 ml = p.ws_ml[part_of(c, r)];
        w = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - mx);
        sum += w * ml.y;
      }
      const int n = min(32, (c1 - cb) / SPLIT + 1);
      for (int i = 0; i < n; i += 16) {  // sixteen parts in flight
        Vec y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (i + e < n) y[e] = load(cb + (i + e) * SPLIT, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (i + e >= n) break;
          const float we = __shfl_sync(0xffffffffu, w, i + e);
          if (we != 0.f) add(acc, we, y[e]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (WAY == kJoinFew) {  // the warps' sums
#pragma unroll
      for (int i = 0; i < kPer; ++i) s_acc[warp][lane * kPer + i] = acc[i];
      if (lane == 0) s_ml[warp] = make_float2(mx, sum);
      __syncthreads();
      if (warp != 0) return;
      mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < SPLIT; ++w) mx = fmaxf(mx, s_ml[w].x);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < SPLIT; ++w) {
        const float2 ml = s_ml[w];
        const float f = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - mx);
        sum += f * ml.y;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += f * s_acc[w][lane * kPer + i];
      }
    }
    finish(r, mx, sum, acc, lane == 0);
  }
}

template <int D, class Plan>
cudaError_t launch_join(const CacheAttnParams& p, int grid, cudaStream_t stream) {
  const int mt_max = row_tiles(p, p.c.max_new);
  const long long tiles = static_cast<long long>(p.c.n_seq) * p.c.hkv * mt_max;
  const bool wide = p.wide;
  // A row a block where a tile has many parts on average, which the other kind reads one
  // after the other, or where there are few such blocks for the GPU (GPU time of a whole
  // call, so and otherwise: 8 tiles of 48 rows in 152 parts 21 and 34 us at d = 128; 64
  // tiles of 4 rows 19 and 23 us at d = 64, 23 and 24 us at 128; 256 tiles of 4 rows 57
  // and 52 us at 128; 32 tiles of 32 rows 22 and 20 us at 128, 16 and 20 us at 64).
  const bool row_a_block = !wide && (tiles * D <= 8ll * p.hg * grid || tiles * p.rows * D <= 128ll * grid);
  // Where a warp may take a row with all its parts (the 8-bit cache): unless the blocks of a row
  // each fit on the SMs at a time (8 tiles of 240 rows in 19 parts: 26 us a row a block).
  const bool few = row_a_block && (!Plan::kEight || tiles * p.rows <= 4ll * grid);
  const bool eight = Plan::kEight && !few && !wide && (row_a_block || p.rows <= kEightRows);
  // By the ends of the CTAs' ranges where these are far fewer than the tiles, most of which are then
  // no CTA's part (a whole call with 8 key heads in 152 ranges, so and otherwise: 200 sequences 56 and
  // 55 us, 512 57 and 63, 1216 60 and 88).
  const bool ends = Plan::kEight && grid > 1 && tiles > 2ll * (grid - 1) * p.hg;
  const long long blocks = (ends ? (grid - 1) * p.hg : tiles) * (few ? p.rows : eight ? (p.rows + 7) / 8 : (p.rows + 31) / 32);
  // The join starts while the attention kernel runs and waits for its end on the
  // device, which hides its launch.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(blocks));
  cfg.blockDim = dim3(wide ? 128 : 256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (few) return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinFew, Plan>, p, grid, mt_max, ends);
  if constexpr (Plan::kEight)
    if (eight) return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinEight, Plan>, p, grid, mt_max, ends);
  if constexpr (Plan::most_rows(D) > kWideRows)
    if (wide) return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinWide, Plan>, p, grid, mt_max, ends);
  if constexpr (!Plan::kEight || Plan::most_rows(D) > kEightRows)
    return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinRows, Plan>, p, grid, mt_max, ends);
  return cudaErrorInvalidConfiguration;  // (not reached: tiles have no more than most_rows rows)
}

}  // namespace
}  // namespace attn
