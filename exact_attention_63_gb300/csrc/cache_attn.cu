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
#include "cache_join.cuh"

#include <type_traits>

namespace attn {
namespace {

constexpr float kTau = 8.0f;  // log2: a row's reference maximum moves when exceeded by more (p ≤ 2^8)

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
  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums), [&](int s) { return units_of<BlockPlan>(p, s); });
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
      const Segment sg = segment_at<BlockPlan>(p, tab, u, u1);
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
        const Segment sg = segment_at<BlockPlan>(p, tab, u, u1);
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
        const Segment sg = segment_at<BlockPlan>(p, tab, u, u1);
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
        const Segment sg = segment_at<BlockPlan>(p, tab, u, u1);
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
      const Segment sg = segment_at<BlockPlan>(p, tab, u, u1);
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
              const bool wide = p.wide;
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
  return launch_join<D, BlockPlan>(p, a.grid, a.stream);
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnLaunch& a) {
  if (a.p.c.d == 64) return a.tiles == 2 ? launch<64, 2>(a) : launch<64, 1>(a);
  return a.tiles == 2 ? launch<128, 2>(a) : launch<128, 1>(a);
}

}  // namespace attn
