// How attention over a paged cache is divided: the key blocks of a sequence, the units of
// the CTAs, the tree of the new tokens.
#pragma once

#include "cache_device.cuh"

namespace attn {
namespace {

// The key blocks of one sequence: `nfull` full ones, then the cached tail and the
// new tokens (at row `off` of block `db`).
struct KeyPlan {
  int q0, n, len;
  int nfull, tail, off, db;
};
__device__ __forceinline__ KeyPlan key_plan(const CacheAttnParams& p, int s) {
  KeyPlan k;
  const SeqRows r = seq_rows(p.c, s);
  k.q0 = r.q0;
  k.n = min(r.n, p.c.max_new);
  k.len = seq_len(p.c, s);
  k.nfull = k.len >> 7;
  k.tail = k.len & 127;
  const int off = (k.tail + p.piece - 1) & ~(p.piece - 1);
  const bool joined = off + ((k.n + 15) & ~15) <= 128;
  k.off = joined ? off : 0;
  k.db = k.nfull + (joined ? 0 : 1);
  return k;
}
struct BlockPlan {
  static constexpr bool kEight = false;  // (ways of the join that its tiles use)
  static constexpr bool kRuns = false;   // units of more than one key head: p.hg of them
  static constexpr int most_rows(int) { return 256; }  // of a CTA's tiles, by d
  static __device__ __forceinline__ KeyPlan of(const CacheAttnParams& p, int s) { return key_plan(p, s); }
};
// Row tiles that the (token, head of the group) rows of n new tokens make.
__host__ __device__ __forceinline__ int row_tiles(const CacheAttnParams& p, int n) {
  return (n * p.c.group + p.rows - 1) / p.rows;
}

// Key heads of a unit.
template <class Plan>
__device__ __forceinline__ int heads_of(const CacheAttnParams& p) {
  return Plan::kRuns ? p.hg : 1;
}

template <class Plan>
__device__ __forceinline__ int units_of(const CacheAttnParams& p, int s) {
  const KeyPlan k = Plan::of(p, s);
  return k.n == 0 ? 0 : p.c.hkv / heads_of<Plan>(p) * row_tiles(p, k.n) * (k.db + 1);
}

__device__ __forceinline__ int range_start(int units, int cta, int grid) {
  return static_cast<int>(static_cast<long long>(units) * cta / grid);
}

// A CTA's share of one (sequence, run of hg key heads, row tile): blocks [b0, b1).  h: the
// number of the run.
struct Segment {
  int s, h, m, b0, b1;
  KeyPlan k;
};
template <class Plan>
__device__ __forceinline__ Segment segment_at(const CacheAttnParams& p, const int* tab, int u, int u_end) {
  Segment g;
  g.s = find_seq(tab, p.c.n_seq, u);
  g.k = Plan::of(p, g.s);
  const int nb = g.k.db + 1, mt = row_tiles(p, g.k.n);
  const int rem = u - tab[g.s], hm = rem / nb;
  g.b0 = rem - hm * nb;
  g.h = hm / mt;
  g.m = hm - g.h * mt;
  g.b1 = min(nb, g.b0 + (u_end - u));
  return g;
}
__device__ __forceinline__ int cached_in(const KeyPlan& k, int b) {
  return b < k.nfull ? 128 : (b == k.nfull ? k.tail : 0);
}

// The ancestors of token t (each lane its own), itself among them, as a set of bits.
// Lane l follows tokens l, l + 32, …: after k rounds it has the 2^k nearest of each and
// the next one up, so the deepest tree takes 7 rounds of at most 30 shuffles (a walk from
// parent to parent took 4.5 us of 21 for 128 drafted tokens, 12 us for a line of them).
__device__ __forceinline__ void ancestors(const int* parents, int n, int t, int lane, uint32_t (&anc)[4]) {
  int up[4];
  uint32_t set[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int token = 32 * i + lane, x = token < n ? parents[token] : -1;
    up[i] = x < token ? x : -1;
#pragma unroll
    for (int w = 0; w < 4; ++w) set[i][w] = w == i ? 1u << lane : 0u;
  }
  while (__any_sync(0xffffffffu, max(max(up[0], up[1]), max(up[2], up[3])) >= 0)) {
    // From the last tokens on: their sources, of no higher a word, are those of the last round.
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      if (32 * i >= n) continue;
      const bool has = up[i] >= 0;
      const int from = max(up[i], 0);
      int far = -1;
      uint32_t more[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        const int x = __shfl_sync(0xffffffffu, up[j], from & 31);
        const bool here = has && (from >> 5) == j;
        if (here) far = x;
#pragma unroll
        for (int w = 0; w <= j; ++w) {
          const uint32_t y = __shfl_sync(0xffffffffu, set[j][w], from & 31);
          if (here) more[w] = y;
        }
      }
      up[i] = far;
#pragma unroll
      for (int w = 0; w <= i; ++w) set[i][w] |= more[w];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (32 * j >= n) break;
#pragma unroll
    for (int w = 0; w <= j; ++w) {
      const uint32_t y = __shfl_sync(0xffffffffu, set[j][w], t & 31);
      if ((t >> 5) == j) anc[w] = y;
    }
  }
}

}  // namespace
}  // namespace attn
