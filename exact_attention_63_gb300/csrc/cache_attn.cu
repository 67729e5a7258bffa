// Attention of new tokens over a paged cache and over each other.
//
//   s_tj = scale·q_t·k_j over the cached keys j and the new tokens j that are t
//   or an ancestor of t;  O_t = Σ_j exp(s_tj − LSE_t)·v_j,  LSE_t = ln Σ_j exp(s_tj).
//
// The group's query heads share one key head, so the rows of one (sequence, key
// head) are its (token, head of the group) pairs: up to 128 of them make the M
// dimension of both products, and every key and value row is read once for all.
// With few rows the operator is bound by reading k and v from device memory
// (4d bytes a key for 4d·rows flops), with ≥ ~128 rows by the tensor core.
//
// Work units are blocks of 128 keys of one (sequence, key head, row tile), in
// that order.  CTA c of G takes the c-th G-th of all units, whatever sequences
// they belong to, so one long sequence and a ragged batch both fill the SMs
// evenly.  A CTA's range covers whole tiles except at its two ends; there it
// leaves an unnormalised part (O, running maximum, sum) in the workspace, and a
// second kernel joins the parts of a tile in order.  The ranges follow from the
// lengths on the device: the host reads nothing back.
//
// Row tiles: MT = 1, up to 128 rows a sequence and key head: two CTAs share an SM (256
// TMEM columns and under half of its shared memory each), K and V of one block each
// (d = 64: two) in flight, one CTA's copies and MMAs under the other's exponentials.
// MT = 2, more rows: one CTA an SM works on two tiles of 128 rows at once, which share
// every block of K and V, two blocks in flight, one tile's MMAs under the other's
// exponentials (with MT = 1 such a call waits for copies).
//   At d = 128 a tile's TMEM has no room for a P beside S, and a P over S costs a round
// trip to the tensor core and back (P·V's commit → barrier → issuer) before the next S can
// be issued; with whole blocks that set the pace.  So (HALVES) the block is taken in two
// halves of 64 keys, each with an S buffer of its own: S of one half is issued while the
// softmax is on the other.  Trees of up to 60 tokens, 16 sequences of up to 4096, 32 heads
// over 8, d = 128 (us, each step with the ones before): MT = 1 82, MT = 2 in whole blocks 79,
// with parts that lie chunk by chunk 71.5, in halves 66.
//   One thread issues all MMAs at MT = 1; at MT = 2 each tile has one, with HALVES one
// for S, and one thread issues both tiles' P·V (one thread for both tiles' S and P·V: 72 us).
//
// P is rounded to bf16, the type of V, which it is multiplied with (both operands of an MMA
// have one type): of O that costs 0.0023 of relative error against float64, where one
// rounding of the exact result costs 0.0017.  Scores, maxima, sums, O and its parts are fp32.
//
// Warps: 0 loads (TMA boxes of a page's rows, one lane a box), then the issuers, and
// four per tile compute its softmax, one thread a row (TMEM lane).
//
// TMEM columns of a tile (256·tile + …):
// d = 128: S [0,128), with P (bf16) over its first half; O [128,256).
//          S(g+1) is issued once P(g)·V has completed.  HALVES: S of half x at [64x, 64x + 64).
// d = 64:  S [0,128), P [128,192), O [192,256): S(g+1) is issued once the softmax
//          has read S(g).
//
// The last cached block and the new tokens' keys share one block where both fit.
// Rows of V that hold no key of the sequence (behind its end, between the two)
// are zeroed in shared memory: their P is 0, but a stale NaN would spread.
#include "attn_fwd_kernel.cuh"
#include "cache_device.cuh"

#include <type_traits>

namespace attn {
namespace {

constexpr int kWideRows = 64;  // parts of more rows lie chunk by chunk, [D/4][rows][4]
constexpr float kTau = 8.0f;  // log2: a row's reference maximum moves when exceeded by more (p ≤ 2^8)

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
// Row tiles of a CTA (MT · nt tokens) that n new tokens make.
__device__ __forceinline__ int row_tiles(const CacheAttnParams& p, int n) { return (n + p.ntt - 1) / p.ntt; }

__device__ __forceinline__ int units_of(const CacheAttnParams& p, int s) {
  const KeyPlan k = key_plan(p, s);
  return k.n == 0 ? 0 : p.c.hkv * row_tiles(p, k.n) * (k.db + 1);
}

__device__ __forceinline__ int range_start(int units, int cta, int grid) {
  return static_cast<int>(static_cast<long long>(units) * cta / grid);
}

// A CTA's share of one (sequence, key head, row tile): blocks [b0, b1).
struct Segment {
  int s, h, m, b0, b1;
  KeyPlan k;
};
__device__ __forceinline__ Segment segment_at(const CacheAttnParams& p, const int* tab, int u, int u_end) {
  Segment g;
  g.s = find_seq(tab, p.c.n_seq, u);
  g.k = key_plan(p, g.s);
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

template <int D, int MT>
struct CL {
  static constexpr bool kHalf = MT == 2 && D == 128;
  static constexpr int kThreads = MT == 1 ? 192 : 384;
  static constexpr int kSoftmax0 = MT == 1 ? 2 : 4;  // first softmax warp
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2;  // 128 rows of Q, K or V: [half][128 rows][128 B]
  static constexpr int kStages = MT == 2 ? (D == 128 ? 2 : 3) : (D == 128 ? 1 : 2);
  static constexpr uint32_t kQ = 0, kK = MT * kTile, kV = kK + kStages * kTile, kBar = kV + kStages * kTile;
  // q_full, q_empty, k_full[S], k_empty[S], v_full[S], v_empty[S], then a tile's s_full[2], p_full[2], pv_done[2], s_free, done[2]
  static constexpr int kNumBars = 2 + 4 * kStages + 9 * MT;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;       // TMEM base, abort flag
  static constexpr uint32_t kSums = kMisc + 8;                 // one int per warp
  static constexpr uint32_t kTable = (kSums + 48 + 15) & ~15u;
  static constexpr uint32_t kBytes = kTable + 1024;            // + alignment; the table comes on top
  static constexpr uint32_t kColS = 0, kColP = D == 128 ? 0 : 128, kColO = D == 128 ? 128 : 192;
};

template <int D, int MT>
__global__ void __launch_bounds__(CL<D, MT>::kThreads, 3 - MT)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                      const __grid_constant__ CUtensorMap tm_vn, const CacheAttnParams p) {
  using L = CL<D, MT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
  const uint32_t q_full = bars, q_empty = bars + 8;
  auto k_full = [&](int s) { return bars + 8u * (2 + s); };
  auto k_empty = [&](int s) { return bars + 8u * (2 + L::kStages + s); };
  auto v_full = [&](int s) { return bars + 8u * (2 + 2 * L::kStages + s); };
  auto v_empty = [&](int s) { return bars + 8u * (2 + 3 * L::kStages + s); };
  constexpr uint32_t kB = 2 + 4 * L::kStages;
  auto s_full = [&](int i, int x) { return bars + 8u * (kB + 9 * i + x); };  // tile i, half x (0 without halves)
  auto p_full = [&](int i, int x) { return bars + 8u * (kB + 9 * i + 2 + x); };
  auto pv_done = [&](int i, int x) { return bars + 8u * (kB + 9 * i + 4 + x); };
  auto s_free = [&](int i) { return bars + 8u * (kB + 9 * i + 6); };
  auto done = [&](int i, int x) { return bars + 8u * (kB + 9 * i + 7 + x); };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 4);
  int* const tab = reinterpret_cast<int*>(smem + L::kTable);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  // TMEM and barriers are set up while the lengths are on their way.
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 256 * MT);
    tmem_relinquish();
    tc_fence_before();
  }
  if (threadIdx.x == 32) {
    *abort_flag = 0u;
    mbar_init(q_full, 1);
    mbar_init(q_empty, MT);  // (each tile's issuer answers for its own reads)
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), MT);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), L::kHalf ? 1 : MT);
    }
    for (int i = 0; i < MT; ++i) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(s_full(i, x), 1);
        mbar_init(p_full(i, x), 4);
        mbar_init(pv_done(i, x), 1);
        mbar_init(done(i, x), 1);
      }
      mbar_init(s_free(i), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 64) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_kn);
    tma_prefetch_desc(&tm_vn);
  }
  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums), [&](int s) { return units_of(p, s); });
  tc_fence_after();
  const int units = tab[p.c.n_seq];
  if (cta == 0)
    for (int i = threadIdx.x; i <= p.c.n_seq; i += L::kThreads) p.ws_table[i] = tab[i];
  const int grid = min(static_cast<int>(gridDim.x), units);  // CTAs with work: each of them at least one unit
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (cta >= grid) {
    if (warp == 0) tmem_dealloc(*tmem_slot, 256 * MT);
    return;
  }
  const int u0 = range_start(units, cta, grid), u1 = range_start(units, cta + 1, grid);
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (warp == 0) {
    // ============================================================= loader
    // All lanes follow; lane 0 waits and announces the bytes, then lane i < 8
    // copies the i-th piece of cached rows and lane 8 + i the i-th 16 new rows.
    auto waited = [&](uint32_t bar, uint32_t parity) -> bool {
      int ok = 1;
      if (lane == 0) ok = wait_bar(bar, parity, wc);
      return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };
    int g = 0, ns = 0, nq = 0, nk = 0, nv = 0;  // blocks, segments; copies issued of each kind
    bool ok = true;
    const int ps = p.piece;
    for (int u = u0; u < u1 && ok; ++ns) {
      const Segment sg = segment_at(p, tab, u, u1);
      u += sg.b1 - sg.b0;
      ok = waited(q_empty, (ns & 1) ^ 1u);
      if (!ok) break;
      if (lane == 0) {
        const int t0 = sg.m * p.ntt, tiles = MT == 2 && sg.k.n - t0 > p.nt ? 2 : 1;
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(tiles * p.nt * p.c.group) * 128u * L::kHalves);
        for (int i = 0; i < tiles; ++i)
          for (int hf = 0; hf < L::kHalves; ++hf)
            tma_load_4d(base + L::kQ + i * L::kTile + hf * 16384, &tm_q, 64 * hf, 0, sg.h, sg.k.q0 + t0 + i * p.nt, q_full);
      }
      ++nq;
      const int nd = (sg.k.n + 15) >> 4;  // 16-row pieces of new keys
      // Page and slot of this lane's piece; the next block's are fetched early.
      int page = 0, slot = 0;
      auto locate = [&](int b) {
        const int j = (b << 7) + lane * ps;
        const int blk = j / p.c.page_size;
        slot = j - blk * p.c.page_size;
        if (lane * ps < cached_in(sg.k, b)) page = page_for_read(p.c, sg.s, blk);
      };
      locate(sg.b0);
      for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g) {
        const int st = g % L::kStages, ph = (g / L::kStages) & 1;
        const int cv = cached_in(sg.k, b), npc = (cv + ps - 1) / ps, ndb = b == sg.k.db ? nd : 0;
        const uint32_t bytes = static_cast<uint32_t>(npc * ps + ndb * 16) * 128u * L::kHalves;
        const int cur_page = page, cur_slot = slot;
        auto copy = [&](const CUtensorMap* mc, const CUtensorMap* mn, uint32_t dst, uint32_t full) {
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          if (lane < npc) {
            for (int hf = 0; hf < L::kHalves; ++hf)
              tma_load_4d(dst + hf * 16384 + lane * ps * 128, mc, 64 * hf, sg.h, cur_slot, cur_page, full);
          } else if (lane >= 8 && lane - 8 < ndb) {
            const int i = lane - 8;
            for (int hf = 0; hf < L::kHalves; ++hf)
              tma_load_4d(dst + hf * 16384 + (sg.k.off + 16 * i) * 128, mn, 64 * hf, sg.h, sg.k.q0 + 16 * i, 0, full);
          }
          __syncwarp();
        };
        ok = waited(k_empty(st), ph ^ 1u) && !(p.test_flags & 1u);
        if (!ok) break;
        copy(&tm_k, &tm_kn, base + L::kK + st * L::kTile, k_full(st));
        ++nk;
        if (b + 1 < sg.b1) locate(b + 1);
        ok = waited(v_empty(st), ph ^ 1u);
        if (!ok) break;
        copy(&tm_v, &tm_vn, base + L::kV + st * L::kTile, v_full(st));
        ++nv;
      }
    }
    // No copy may be in flight when the CTA ends (the newest of each slot; older ones
    // landed before their slot was filled again).  Another warp's wait may have run out
    // after the last copy was issued, so this does not depend on `ok`.
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      auto drain = [&](uint32_t bar, uint32_t parity) {
        while (!mbar_try_wait(bar, parity))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
      };
      if (nq > 0) drain(q_full, (nq - 1) & 1);
      for (int n = max(0, nk - L::kStages); n < nk; ++n) drain(k_full(n % L::kStages), (n / L::kStages) & 1u);
      for (int n = max(0, nv - L::kStages); n < nv; ++n) drain(v_full(n % L::kStages), (n / L::kStages) & 1u);
    }
  } else if (L::kHalf && warp <= 2) {
    // =============================================== halves: a tile's S issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, 64, false);
      const int tile = warp - 1;
      const uint64_t dq = sdesc_kmajor_sw128(base + L::kQ + tile * L::kTile);
      int g = 0, ns = 0;  // blocks and segments of the CTA
      int e = 0;          // blocks of this tile: fewer, where a segment has rows for the first tile only
      bool ok = true;
      for (int u = u0; u < u1 && ok; ++ns) {
        const Segment sg = segment_at(p, tab, u, u1);
        u += sg.b1 - sg.b0;
        const bool now = tile == 0 || sg.k.n - sg.m * p.ntt > p.nt;
        ok = wait_bar(q_full, ns & 1, wc);
        for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g) {
          const int st = g % L::kStages;
          ok = wait_bar(k_full(st), (g / L::kStages) & 1, wc);
          if (now) {
            const uint64_t dk = sdesc_kmajor_sw128(base + L::kK + st * L::kTile);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              // The half's last product has read its P, which lies over S.
              if (e > 0) ok = ok && wait_bar(pv_done(tile, x), (e - 1) & 1, wc);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                mma_ss(tmem + 256 * tile + 64 * x, dq + o, dk + o + ((x * 8192) >> 4), idS, kk > 0 ? 1u : 0u);
              }
              mma_commit(s_full(tile, x));
            }
            ++e;
          } else {
            // No rows here.  V is waited for all the same: the softmax looks at v_full in
            // some blocks only, and a wait on a parity is right only for the phase after
            // one that is known to be over.  So S of a block is issued when V of all
            // blocks before it is known to have arrived: by this wait, or by the product
            // of this tile's last block.
            if (e > 0) ok = ok && wait_bar(pv_done(tile, 1), (e - 1) & 1, wc);
            ok = ok && wait_bar(v_full(st), (g / L::kStages) & 1, wc);
          }
          if (!ok) break;
          mma_commit(k_empty(st));
          if (b == sg.b1 - 1) mma_commit(q_empty);
        }
      }
      mma_commit(done(tile, 0));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(done(tile, 0), 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
  } else if (L::kHalf && warp == 3) {
    // ============================================ halves: both tiles' P·V issuer
    if (lane == 0) {
      constexpr uint32_t idPV = idesc_bf16(128, D, true);
      int g = 0, e1 = 0;  // blocks of the CTA (and of the first tile), blocks of the second
      bool ok = true;
      for (int u = u0; u < u1 && ok;) {
        const Segment sg = segment_at(p, tab, u, u1);
        u += sg.b1 - sg.b0;
        const int tiles = sg.k.n - sg.m * p.ntt > p.nt ? 2 : 1;
        for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g) {
          const int st = g % L::kStages;
          ok = wait_bar(v_full(st), (g / L::kStages) & 1, wc);
          const uint64_t dv = sdesc_mnmajor_sw128(base + L::kV + st * L::kTile, 16384);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            for (int i = 0; i < tiles; ++i) {
              ok = ok && wait_bar(p_full(i, x), (i == 0 ? g : e1) & 1, wc);
              if (!ok) break;
              tc_fence_after();
              const uint32_t t = tmem + 256 * i;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(t + L::kColO, t + 64 * x + kk * 8, dv + (((4 * x + kk) * 2048) >> 4), idPV,
                       (b > sg.b0 || x > 0 || kk > 0) ? 1u : 0u);
              mma_commit(pv_done(i, x));
            }
          if (!ok) break;
          mma_commit(v_empty(st));
          if (tiles == 2) ++e1;
        }
      }
      mma_commit(done(0, 1));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(done(0, 1), 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
  } else if (!L::kHalf && warp <= MT) {
    // ==================================================== a tile's MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, 128, false);
      constexpr uint32_t idPV = idesc_bf16(128, D, true);
      const int tile = warp - 1;
      const uint32_t t = tmem + 256 * tile;
      int g = 0, ns = 0, e = 0;  // as above
      bool before = false;       // this tile's product of block g − 1 is to come
      bool first = false;        // which opens its segment
      bool ok = true;
      // O (+)= P·V of block g − 1.
      auto issue_pv = [&]() -> bool {
        const int st = (g - 1) % L::kStages;
        if (!wait_bar(v_full(st), ((g - 1) / L::kStages) & 1, wc) || !wait_bar(p_full(tile, 0), (e - 1) & 1, wc))
          return false;
        tc_fence_after();
        const uint64_t dv = sdesc_mnmajor_sw128(base + L::kV + st * L::kTile, 16384);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(t + L::kColO, t + L::kColP + kk * 8, dv + ((kk * 2048) >> 4), idPV, (!first || kk > 0) ? 1u : 0u);
        mma_commit(pv_done(tile, 0));
        mma_commit(v_empty(st));
        return true;
      };
      for (int u = u0; u < u1 && ok; ++ns) {
        const Segment sg = segment_at(p, tab, u, u1);
        u += sg.b1 - sg.b0;
        const bool now = tile == 0 || sg.k.n - sg.m * p.ntt > p.nt;
        for (int b = sg.b0; b < sg.b1; ++b, ++g) {
          const int st = g % L::kStages;
          if (D == 128 && before) ok = ok && issue_pv();  // the last P lies over S: its product has to be done first
          if (b == sg.b0) ok = ok && wait_bar(q_full, ns & 1, wc);
          ok = ok && wait_bar(k_full(st), (g / L::kStages) & 1, wc);
          if (now && e > 0)
            ok = ok && (D == 128 ? wait_bar(pv_done(tile, 0), (e - 1) & 1, wc) : wait_bar(s_free(tile), (e - 1) & 1, wc));
          if (!ok) break;
          if (now) {
            tc_fence_after();
            const uint64_t dq = sdesc_kmajor_sw128(base + L::kQ + tile * L::kTile);
            const uint64_t dk = sdesc_kmajor_sw128(base + L::kK + st * L::kTile);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
              mma_ss(t + L::kColS, dq + o, dk + o, idS, kk > 0 ? 1u : 0u);
            }
            mma_commit(s_full(tile, 0));
          }
          mma_commit(k_empty(st));
          if (b == sg.b1 - 1) mma_commit(q_empty);
          if (D == 64 && before) ok = issue_pv();
          if (!ok) break;
          if (MT == 2 && !now) {  // no product of this block here
            ok = wait_bar(v_full(st), (g / L::kStages) & 1, wc);
            if (!ok) break;
            mma_commit(v_empty(st));
          }
          before = now;
          first = b == sg.b0;
          e += now;
        }
      }
      if (ok && before) issue_pv();
      mma_commit(done(tile, 0));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(done(tile, 0), 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
  } else if (warp >= L::kSoftmax0 && warp < L::kSoftmax0 + 4 * MT) {
    // ============================================================ softmax
    const int tile = MT == 1 ? 0 : (warp - L::kSoftmax0) >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_base = tmem + 256 * tile + lane_off;
    const uint32_t tS = t_base + L::kColS, tP = t_base + L::kColP, tO = t_base + L::kColO;
    const float sc = p.scale_log2;
    const uint64_t sc2 = pack2(sc, sc);
    int g = 0, e = 0;  // blocks of the CTA and of this tile, as the issuer counts them
    bool ok = true;
    for (int u = u0; u < u1 && ok;) {
      const Segment sg = segment_at(p, tab, u, u1);
      const bool first_of_cta = u == u0;
      u += sg.b1 - sg.b0;
      const int t0 = sg.m * p.ntt + tile * p.nt, n_rows = min(sg.k.n - t0, p.nt) * p.c.group;
      if (MT == 2 && n_rows <= 0) {
        g += sg.b1 - sg.b0;
        continue;
      }
      const bool active = (warp & 3) * 32 < n_rows;
      float m_run = -INFINITY, l_run = 0.f;
      uint32_t anc[4] = {0u, 0u, 0u, 0u};  // the new tokens this row sees
      if (sg.b1 > sg.k.db && active) {
        const int t = min(t0 + r / p.c.group, sg.k.n - 1);
        if (p.parents == nullptr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int bits = min(max(t + 1 - 32 * i, 0), 32);
            anc[i] = bits == 32 ? 0xffffffffu : (1u << bits) - 1u;
          }
        } else {
          ancestors(p.parents + sg.k.q0, sg.k.n, t, lane, anc);
        }
      }
      // A block's keys, or half x of them.
      constexpr int kCh = L::kHalf ? 2 : 4;  // chunks of 32 keys
      auto block = [&](int b, int x, auto mask_tag) -> bool {
        constexpr bool MASK = decltype(mask_tag)::value;
        const uint32_t tSx = tS + 64 * x, tPx = L::kHalf ? tSx : tP;
        const bool got = wait_bar_cold(s_full(tile, x), e & 1, wc);
        if (__any_sync(0xffffffffu, !got)) return false;
        tc_fence_after();
        uint32_t vis[kCh];
        if constexpr (MASK) {
          const int cv = cached_in(sg.k, b), dn = b == sg.k.db ? sg.k.n : 0;
          const int sh = sg.k.off >> 5, bit = sg.k.off & 31;
#pragma unroll
          for (int c = 0; c < kCh; ++c) {
            const int cc = c + 2 * x;
            const int n = min(max(cv - 32 * cc, 0), 32);
            vis[c] = n == 32 ? 0xffffffffu : (1u << n) - 1u;
            if (dn > 0) {
              uint32_t lo = 0u, hi = 0u;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i == cc - sh) hi = anc[i];
                if (i == cc - sh - 1) lo = anc[i];
              }
              vis[c] |= __funnelshift_l(lo, hi, bit);
            }
          }
          if (x == 0) {
            // Zero the rows of V that hold no key (every warp its 32 rows).
            const int st = g % L::kStages;
            const bool in = wait_bar_cold(v_full(st), (g / L::kStages) & 1, wc);
            if (__any_sync(0xffffffffu, !in)) return false;
            if (!(r < cv || (r >= sg.k.off && r < sg.k.off + dn))) {
              uint8_t* const row = smem + L::kV + st * L::kTile + r * 128;
#pragma unroll
              for (int i = 0; i < 8 * L::kHalves; ++i)
                *reinterpret_cast<uint4*>(row + (i >> 3) * 16384 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (active) {
          uint32_t a[32], c2[32];
          float mx = -INFINITY;
          // ---- maximum
          if constexpr (MASK) {
#pragma unroll
            for (int c = 0; c < kCh; c += 2) {
              tmem_ld32(tSx + 32 * c, a);
              tmem_ld32(tSx + 32 * c + 32, c2);
              tmem_wait_ld();
              reg_fence32(a);
              reg_fence32(c2);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if ((vis[c] >> i) & 1u) mx = fmaxf(mx, __uint_as_float(a[i]));
                if ((vis[c + 1] >> i) & 1u) mx = fmaxf(mx, __uint_as_float(c2[i]));
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < kCh; c += 2) {
              float m0, m1;
              tmem_ld32_max(tSx + 32 * c, a, m0);
              tmem_ld32_max(tSx + 32 * c + 32, c2, m1);
              tmem_wait_ld();
              asm volatile("" : "+f"(m0), "+f"(m1));
              reg_fence32(a);
              reg_fence32(c2);
              mx = fmax3(mx, m0, m1);
            }
          }
          mx *= sc;
          const bool need = r < n_rows && (mx > m_run + kTau || (m_run == -INFINITY && mx > -INFINITY));
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = need ? mx : m_run;
            if (b > sg.b0 || x > 0) {
              const float alpha = need ? ex2_mufu(m_run - m_new) : 1.f;
              // (the product before this one: the other half's, or the last block's)
              const uint32_t bar = pv_done(tile, L::kHalf ? x ^ 1 : 0), par = (x > 0 ? e : e - 1) & 1;
              if constexpr (L::kHalf) {  // in line: a call would have to put the scores away
                const bool landed = wait_bar(bar, par, wc);
                if (__any_sync(0xffffffffu, !landed)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t o[16];
                  tmem_ld16(tO + 16 * c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+r"(o[i]));
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                  }
                  tmem_st16(tO + 16 * c, o);
                }
              } else {
                if (!rescale_o<D>(bar, par, wc, tO, alpha)) return false;
              }
              l_run *= alpha;
            }
            m_run = m_new;
          }
          // ---- exponentials, P in bf16
          if constexpr (D == 64) {
            if (e > 0) {  // the last P·V has read P
              const bool landed = wait_bar_cold(pv_done(tile, 0), (e - 1) & 1, wc);
              if (__any_sync(0xffffffffu, !landed)) return false;
              tc_fence_after();
            }
          }
          const float negm = m_run == -INFINITY ? 0.f : -m_run;
          const uint64_t nm2 = pack2(negm, negm);
          uint64_t acc[2] = {0, 0};
          auto chunk = [&](int c, uint32_t(&v)[32]) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1;
              unpack2(ffma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2, nm2), x0, x1);
              x0 = ex2_mufu(x0);
              x1 = ex2_mufu(x1);
              if constexpr (MASK) {
                x0 = (vis[c] >> (2 * i)) & 1u ? x0 : 0.f;
                x1 = (vis[c] >> (2 * i + 1)) & 1u ? x1 : 0.f;
              }
              acc[i & 1] = fadd2(acc[i & 1], pack2(x0, x1));
              pk[i] = pack_bf16x2(x0, x1);
            }
            tmem_st16(tPx + 16 * c, pk);
          };
          if constexpr (L::kHalf) {  // a half's scores are in registers since the maximum
            chunk(0, a);
            chunk(1, c2);
          } else {
            tmem_ld32(tSx, a);
#pragma unroll
            for (int c = 0; c < kCh; c += 2) {
              tmem_wait_ld();
              reg_fence32(a);
              tmem_ld32(tSx + 32 * (c + 1), c2);
              chunk(c, a);
              tmem_wait_ld();
              reg_fence32(c2);
              if (c + 2 < kCh) tmem_ld32(tSx + 32 * (c + 2), a);
              chunk(c + 1, c2);
            }
          }
          float a0, a1;
          unpack2(fadd2(acc[0], acc[1]), a0, a1);
          l_run += a0 + a1;
          tmem_wait_st();
        }
        tc_fence_before();
        if constexpr (D == 64) warp_arrive(s_free(tile), lane);
        warp_arrive(p_full(tile, x), lane);
        return true;
      };
      for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g, ++e)
#pragma unroll 1
        for (int x = 0; x < (L::kHalf ? 2 : 1) && ok; ++x)
          ok = b < sg.k.nfull ? block(b, x, std::false_type{}) : block(b, x, std::true_type{});
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (active) {
        const bool landed = wait_bar_cold(pv_done(tile, L::kHalf), (e - 1) & 1, wc);
        if (__any_sync(0xffffffffu, !landed)) { ok = false; break; }
        tc_fence_after();
        const bool whole = sg.b0 == 0 && sg.b1 == sg.k.db + 1;
        const int grp = p.c.group, t = t0 + r / grp, hq = sg.h * grp + r % grp, H = p.c.hkv * grp;
        const long long token = sg.k.q0 + t;
        const int slot = 2 * cta + (first_of_cta ? 0 : 1);
        const long long part = static_cast<long long>(slot) * p.rows + tile * p.nt * grp + r;
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(tO + 32 * c, x);
          tmem_wait_ld();
          reg_fence32(x);
          if (r < n_rows) {
            if (whole) {
              uint4* const dst = reinterpret_cast<uint4*>(p.o + (token * H + hq) * D + 32 * c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t* o8 = &x[8 * i];
                uint4 w;
                w.x = pack_bf16x2(__uint_as_float(o8[0]) * inv, __uint_as_float(o8[1]) * inv);
                w.y = pack_bf16x2(__uint_as_float(o8[2]) * inv, __uint_as_float(o8[3]) * inv);
                w.z = pack_bf16x2(__uint_as_float(o8[4]) * inv, __uint_as_float(o8[5]) * inv);
                w.w = pack_bf16x2(__uint_as_float(o8[6]) * inv, __uint_as_float(o8[7]) * inv);
                dst[i] = w;
              }
            } else {
              // Row by row, or (many rows) four values of every row side by side, so
              // that a warp's store is one run of bytes: as 32 pieces of 16 bytes the
              // parts of a tile of 256 rows took 6 us to leave the SM.
              const bool wide = p.rows > kWideRows;
              uint4* dst = reinterpret_cast<uint4*>(p.ws_o) +
                           (wide ? (static_cast<long long>(slot) * (D / 4) + 8 * c) * p.rows + tile * p.nt * grp + r
                                 : part * (D / 4) + 8 * c);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                *dst = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                dst += wide ? p.rows : 1;
              }
            }
          }
        }
        if (r < n_rows) {
          if (whole)
            p.lse[static_cast<long long>(hq) * p.c.total + token] =
                l_run == 0.f ? -INFINITY : (m_run + __log2f(l_run)) * 0.69314718055994531f;
          else
            p.ws_ml[part] = make_float2(m_run, l_run);
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256 * MT);
  }
}

// Joins the parts of the tiles that were split.  With the parts' maxima m_i and
// sums l_i:  m = max m_i,  O = Σ 2^(m_i − m) O_i / Σ 2^(m_i − m) l_i.
// WAY = kJoinFew: a block takes one row, its eight warps deal out the parts (few rows;
// one long sequence leaves a part on every CTA).  kJoinRows: a block takes 32 rows, a
// warp four at once.  kJoinWide: parts that lie chunk by chunk; a block takes 32 rows,
// a lane a row, a warp a quarter of its values.
enum { kJoinFew, kJoinRows, kJoinWide };

template <int D, int WAY>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttnParams p, int grid, int mt_max) {
  constexpr int kPer = D / 32, SPLIT = 8;
  __shared__ float s_acc[WAY == kJoinFew ? SPLIT : 1][D];
  __shared__ float2 s_ml[SPLIT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned int chunks = WAY == kJoinFew ? p.rows : (p.rows + 31) / 32;
  unsigned int x = blockIdx.x;
  const int row0 = static_cast<int>(x % chunks) * (WAY == kJoinFew ? 1 : 32);
  x /= chunks;
  const int m = static_cast<int>(x % mt_max);
  x /= mt_max;
  const int h = static_cast<int>(x % p.c.hkv), s = static_cast<int>(x / p.c.hkv);
  const KeyPlan k = key_plan(p, s);
  const int grp = p.c.group, t0 = m * p.ntt, n_rows = min(k.n - t0, p.ntt) * grp;
  // The attention kernel's results, complete and visible.  Every block waits, so
  // that this kernel never ends before that one.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row0 >= n_rows) return;
  const int units = p.ws_table[p.c.n_seq], nb = k.db + 1;
  grid = min(grid, units);
  const int ua = p.ws_table[s] + (h * row_tiles(p, k.n) + m) * nb;
  auto cta_of = [&](int u) { return static_cast<int>(((u + 1ll) * grid - 1) / units); };
  const int c0 = cta_of(ua), c1 = cta_of(ua + nb - 1);
  if (c0 == c1) return;  // one CTA did it all and has written the rows
  // Every CTA's part but the first's is the first of its range.
  const int slot0 = 2 * c0 + (range_start(units, c0, grid) >= ua ? 0 : 1);
  auto part_of = [&](int c, int r) { return static_cast<long long>(c == c0 ? slot0 : 2 * c) * p.rows + r; };

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
    const int hq = h * grp + r % grp;
    const long long token = k.q0 + t0 + r / grp;
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
                          (static_cast<long long>(c == c0 ? slot0 : 2 * c) * (D / 4) + first) * p.rows + r;
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
    const int hq = h * grp + r % grp;
    const long long token = k.q0 + t0 + r / grp;
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
    const int r = row0;
    float mx = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int c = c0 + warp + lane * SPLIT; c <= c1; c += 32 * SPLIT) mx = fmaxf(mx, p.ws_ml[part_of(c, r)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    for (int cb = c0 + warp; cb <= c1; cb += 32 * SPLIT) {
      const int c = cb + lane * SPLIT;
      float w = 0.f;
      if (c <= c1) {
        const float2 ml = p.ws_ml[part_of(c, r)];
        w = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - mx);
        sum += w * ml.y;
      }
      const int n = min(32, (c1 - cb) / SPLIT + 1);
      for (int i = 0; i < n; i += 16) {  // sixteen parts in flight; behind the last, weight 0
        Vec y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = load(min(cb + (i + e) * SPLIT, c1), r);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float we = __shfl_sync(0xffffffffu, w, i + e);
          if (we != 0.f) add(acc, we, y[e]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
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
    finish(r, mx, sum, acc, lane == 0);
  }
}

template <int D, int MT>
cudaError_t launch(const CacheAttnLaunch& a) {
  using L = CL<D, MT>;
  const CacheAttnParams& p = a.p;
  const unsigned int smem = L::kBytes + 4u * (p.c.n_seq + 1);
  static volatile bool configured[64] = {};
  if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
  if (!configured[a.device]) {
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               L::kBytes + 4 * (kCacheMaxSeq + 1));
    if (e != cudaSuccess) return e;
    configured[a.device] = true;
  }
  cache_attn_kernel<D, MT><<<a.grid, L::kThreads, smem, a.stream>>>(a.q, a.k, a.v, a.kn, a.vn, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int mt_max = (p.c.max_new + p.ntt - 1) / p.ntt;
  const long long tiles = static_cast<long long>(p.c.n_seq) * p.c.hkv * mt_max;
  const bool wide = p.rows > kWideRows;
  // A row a block where a tile has many parts on average, which the other kind reads one
  // after the other, or where there are few such blocks for the GPU (GPU time of a whole
  // call, so and otherwise: 8 tiles of 48 rows in 152 parts 21 and 34 us at d = 128; 64
  // tiles of 4 rows 19 and 23 us at d = 64, 23 and 24 us at 128; 256 tiles of 4 rows 57
  // and 52 us at 128; 32 tiles of 32 rows 22 and 20 us at 128, 16 and 20 us at 64).
  const bool few = !wide && (tiles * D <= 8ll * a.grid || tiles * p.rows * D <= 128ll * a.grid);
  const long long blocks = tiles * (few ? p.rows : (p.rows + 31) / 32);
  // The join starts while the attention kernel runs and waits for its end on the
  // device, which hides its launch.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(blocks));
  cfg.blockDim = dim3(wide ? 128 : 256);
  cfg.stream = a.stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (wide) return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinWide>, p, a.grid, mt_max);
  return few ? cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinFew>, p, a.grid, mt_max)
             : cudaLaunchKernelEx(&cfg, cache_join_kernel<D, kJoinRows>, p, a.grid, mt_max);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnLaunch& a) {
  if (a.p.c.d == 64) return a.tiles == 2 ? launch<64, 2>(a) : launch<64, 1>(a);
  return a.tiles == 2 ? launch<128, 2>(a) : launch<128, 1>(a);
}

}  // namespace attn
