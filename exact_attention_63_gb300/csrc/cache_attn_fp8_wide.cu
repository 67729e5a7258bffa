// Attention of new tokens over a paged cache of E4M3 codes and over each other, many rows
// (cache_attn_fp8.cu has the formulas, and the kernel for few).
//
// With more than 16 rows a sequence and key head (d = 64: 32) the products belong on the tensor core's
// tcgen05 instructions, whose operands have 16 bits: 8 or 16 warps (the converters) read the
// codes, 16 bytes a lane and whole rows of a head at a time, take them to bf16 with their
// scales, which is exact, and lay them out in shared memory as TMA would; all that follows is as over a
// cache of bf16 (cache_attn.cu): S of 64 keys at a time, the softmax of one row a thread with P over
// S, O in tensor memory, units of 128 keys dealt out evenly, parts joined by a second kernel.
//   Each code costs the converters about three instructions and the shared memory 4 bytes
// (written once, read once), half of what its 128 bytes a cycle carry in the time that
// memory takes to deliver it.  A run's registers take the codes that come next (K's, V's, the next
// block's K's) as soon as it is converted, so memory is at work under products and exponentials.
//
// Row tiles: MT = 1, up to 128 rows a sequence and key head: two CTAs share an SM (256 TMEM columns
// each).  MT = 2, more rows: one CTA an SM has two tiles of 128, which share every block the
// converters lay out, two blocks of K and V at a time.
// Warps: 0 and 1 load a tile's Q (TMA) and issue its S, 2 issues both tiles' P·V, 3 looks up what
// the converters copy (pages, scales, new tokens; four units at a time and up to twelve ahead,
// so that nobody waits for a page table); then four a tile for the softmax and the converters: 8, or with
// MT = 2 16 (64 tokens over 64 sequences of up to 8191: 352 us, with 8 of them 396).
//   The registers are split between the roles.  Next to nothing may spill: shared memory takes up nearly all
// of L1, so a reload comes from L2, and in the chain product, softmax, product it shows (with the issuers at
// 40 registers instead of 56 the trees took 74 us instead of 70, 64 tokens 444 instead of 412).
//
// TMEM columns of a tile (256·tile + …): S of half x of a block at [64x, 64x + 64), P (bf16) over
// its first half; O [128, 128 + d).
#include "attn_fwd_kernel.cuh"
#include "cache_join.cuh"
#include "fp8_device.cuh"

#include <type_traits>

namespace attn {
namespace {

constexpr float kTau = 8.0f;  // log2: a row's reference maximum moves when exceeded by more (p ≤ 2^8)
// Registers a thread of the issuers' warpgroup, the softmax's (MT of them) and the converters'
// (two or four); together no more than what the block is launched with.  (MT = 1 with 24, 120 and 56:
// 278 us instead of 240 for 16 tokens over 64 sequences; with 40, 120 and 48: 269.)
template <int MT>
struct Regs {
  static constexpr int kConverters = MT == 1 ? 8 : 16;
  static constexpr int kLaunch = MT == 1 ? 64 : 72, kIssuer = MT == 1 ? 32 : 56, kSoftmax = MT == 1 ? 112 : 128,
                       kConverter = MT == 1 ? 56 : 48;
  static_assert(kIssuer + MT * kSoftmax + kConverters / 4 * kConverter <= (1 + MT + kConverters / 4) * kLaunch,
                "the split has to fit");
};

// The blocks of the bf16 cache's kernel.
struct ConvertPlan {
  static constexpr bool kEight = true, kRuns = false;
  static constexpr int most_rows(int) { return 256; }
  static __device__ __forceinline__ KeyPlan of(const CacheAttnParams& p, int s) { return key_plan(p, s); }
};

struct CacheAttnFp8WideParams {
  CacheAttnParams a;
  Fp8Pages f;
  const uint16_t* kn;
  const uint16_t* vn;
  long long kn_st[2], vn_st[2];
};

// What the converters have to know of a unit: its 16 slots' places in the cache (−1: no key)
// and scales, how many keys are the cache's, and where the new tokens' lie.
struct Unit {
  long long k_at[8], v_at[8];     // bytes
  float k_scale[8], v_scale[8];
  int cached, off, fresh, q0, h;
  int pad[3];
};
constexpr int kBatches = 4;       // of four units each

template <int D, int MT>
struct WL {
  static constexpr int kConverter0 = 4 + 4 * MT;   // first converter warp
  static constexpr int kConverters = Regs<MT>::kConverters;
  static constexpr int kThreads = 32 * (kConverter0 + kConverters);
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2;  // 128 rows of Q, K or V: [half][128 rows][128 B]
  static constexpr int kStages = D == 128 && MT == 1 ? 1 : 2;
  static constexpr uint32_t kQ = 0, kK = MT * kTile, kV = kK + kStages * kTile, kBar = kV + kStages * kTile;
  // k_full[S], k_empty[S], v_full[S], v_empty[S], u_full[kBatches], u_empty[kBatches], then a tile's q_full,
  // q_empty, s_full[2], p_full[2], pv_done[2], done; pv_end
  static constexpr int kNumBars = 4 * kStages + 2 * kBatches + 9 * MT + 1;
  static constexpr uint32_t kUnits = (kBar + 8 * kNumBars + 15) & ~15u;  // [batch][4] Unit
  static constexpr uint32_t kMisc = kUnits + kBatches * 4 * sizeof(Unit);  // TMEM base, abort flag
  static constexpr uint32_t kSums = kMisc + 8;            // one int per warp
  static constexpr uint32_t kTable = (kSums + kThreads / 8 + 15) & ~15u;
  static constexpr uint32_t kBytes = kTable + 1024;       // + alignment; the table comes on top
  static constexpr uint32_t kColO = 128;
};

// 16 codes (a run of a row) times 2^(e − 127) as bf16, exactly.
__device__ __forceinline__ void to_bf16(const uint4& codes, float f, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const uint64_t f2 = pack2(f, f);
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    f16x2_to_f32(e4m3x2_to_f16x2(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]), a, b);
    unpack2(fmul2(pack2(a, b), f2), a, b);
    out[i] = pack_bf16x2(a, b);
  }
  lo = make_uint4(out[0], out[1], out[2], out[3]);
  hi = make_uint4(out[4], out[5], out[6], out[7]);
}

// wait_bar for roles with few registers: the flag by its 32-bit address.
__device__ __forceinline__ bool wait_few(uint32_t bar, uint32_t parity, uint32_t flag, const CacheAttnParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15) == 0) {
      uint32_t set;
      asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(set) : "r"(flag) : "memory");
      if (set) return false;
      if (globaltimer_ns() - t0 > p.timeout_ns) {
        asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(flag), "r"(1u) : "memory");
        atomicOr(p.status, kStatusTimeout);
        return false;
      }
    }
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(WL<D, MT>::kThreads, 3 - MT)
    cache_attn_fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const CacheAttnFp8WideParams fp) {
  using L = WL<D, MT>;
  using R = Regs<MT>;
  const CacheAttnParams& p = fp.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
  auto k_full = [&](int s) { return bars + 8u * s; };
  auto k_empty = [&](int s) { return bars + 8u * (L::kStages + s); };
  auto v_full = [&](int s) { return bars + 8u * (2 * L::kStages + s); };
  auto v_empty = [&](int s) { return bars + 8u * (3 * L::kStages + s); };
  auto u_full = [&](int i) { return bars + 8u * (4 * L::kStages + i); };
  auto u_empty = [&](int i) { return bars + 8u * (4 * L::kStages + kBatches + i); };
  constexpr uint32_t kB = 4 * L::kStages + 2 * kBatches;
  auto q_full = [&](int i) { return bars + 8u * (kB + 9 * i); };  // of tile i
  auto q_empty = [&](int i) { return bars + 8u * (kB + 9 * i + 1); };
  auto s_full = [&](int i, int x) { return bars + 8u * (kB + 9 * i + 2 + x); };
  auto p_full = [&](int i, int x) { return bars + 8u * (kB + 9 * i + 4 + x); };
  auto pv_done = [&](int i, int x) { return bars + 8u * (kB + 9 * i + 6 + x); };
  auto done = [&](int i) { return bars + 8u * (kB + 9 * i + 8); };
  const uint32_t pv_end = bars + 8u * (kB + 9 * MT);
  Unit* const found = reinterpret_cast<Unit*>(smem + L::kUnits);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 4);
  int* const tab = reinterpret_cast<int*>(smem + L::kTable);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 256 * MT);
    tmem_relinquish();
    tc_fence_before();
  }
  if (threadIdx.x == 32) {
    *abort_flag = 0u;
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(k_full(s), L::kConverters);
      mbar_init(k_empty(s), MT);  // (each tile's issuer answers for its own reads)
      mbar_init(v_full(s), L::kConverters);
      mbar_init(v_empty(s), 1);
    }
    for (int i = 0; i < kBatches; ++i) {
      mbar_init(u_full(i), 1);
      mbar_init(u_empty(i), L::kConverters);
    }
    for (int i = 0; i < MT; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(s_full(i, x), 1);
        mbar_init(p_full(i, x), 4);
        mbar_init(pv_done(i, x), 1);
      }
      mbar_init(done(i), 1);
    }
    mbar_init(pv_end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 64) tma_prefetch_desc(&tm_q);
  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums),
               [&](int s) { return units_of<ConvertPlan>(p, s); });
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

  const uint32_t flag = base + L::kMisc + 4;  // abort_flag
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kIssuer));
    if (lane == 0 && warp < MT) {
      // ================================================ a tile's Q and S
      constexpr uint32_t idS = idesc_bf16(128, 64, false);
      const int tile = MT == 1 ? 0 : warp;
      const uint32_t q_at = base + L::kQ + tile * L::kTile;
      const uint64_t dq = sdesc_kmajor_sw128(q_at);
      int g = 0, nq = 0, e = 0;  // blocks of the CTA; copies of Q; blocks of this tile (fewer, where a segment has rows for the first only)
      bool ok = true;
      for (int u = u0; u < u1 && ok;) {
        const Segment sg = segment_at<ConvertPlan>(p, tab, u, u1);
        u += sg.b1 - sg.b0;
        const int t0 = sg.m * p.ntt + tile * p.nt;
        const bool now = tile == 0 || sg.k.n > t0;
        if (now) {
          ok = nq == 0 || wait_few(q_empty(tile), (nq - 1) & 1, flag, p);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full(tile), static_cast<uint32_t>(p.nt * p.c.group) * 128u * L::kHalves);
          for (int hf = 0; hf < L::kHalves; ++hf)
            tma_load_4d(q_at + hf * 16384, &tm_q, 64 * hf, 0, sg.h, sg.k.q0 + t0, q_full(tile));
          ok = wait_few(q_full(tile), nq & 1, flag, p);
          ++nq;
        }
        for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g) {
          const int st = g % L::kStages;
          ok = wait_few(k_full(st), (g / L::kStages) & 1, flag, p);
          if (!ok) break;
          if (now) {
            const uint64_t dk = sdesc_kmajor_sw128(base + L::kK + st * L::kTile);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              // The half's last product has read its P, which lies over S.
              if (e > 0) ok = ok && wait_few(pv_done(tile, x), (e - 1) & 1, flag, p);
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
            if (!ok) break;
            if (b == sg.b1 - 1) mma_commit(q_empty(tile));
          }
          mma_commit(k_empty(st));
        }
      }
      mma_commit(done(tile));
      // No product and no copy may be in flight when the CTA ends, whatever ended the loop.
      const uint64_t t0 = globaltimer_ns();
      auto drain = [&](uint32_t bar, uint32_t parity) {
        while (!mbar_try_wait(bar, parity))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
      };
      drain(done(tile), 0);
      if (nq > 0) drain(q_full(tile), (nq - 1) & 1);
    } else if (lane == 0 && warp == 2) {
      // ==================================================== P·V of all tiles
      constexpr uint32_t idPV = idesc_bf16(128, D, true);
      int g = 0, e1 = 0;  // blocks of the CTA (and of the first tile), blocks of the second
      bool ok = true;
      for (int u = u0; u < u1 && ok;) {
        const Segment sg = segment_at<ConvertPlan>(p, tab, u, u1);
        u += sg.b1 - sg.b0;
        const int tiles = MT == 2 && sg.k.n - sg.m * p.ntt > p.nt ? 2 : 1;
        for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g) {
          const int st = g % L::kStages;
          ok = wait_few(v_full(st), (g / L::kStages) & 1, flag, p);
          const uint64_t dv = sdesc_mnmajor_sw128(base + L::kV + st * L::kTile, 16384);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            for (int i = 0; i < tiles; ++i) {
              ok = ok && wait_few(p_full(i, x), (i == 0 ? g : e1) & 1, flag, p);
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
      mma_commit(pv_end);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(pv_end, 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
    if (warp == 3) {
      // ======================================================== look-ups
      // Lane 8q + i: the i-th 16 slots of the q-th unit of a batch.
      bool ok = true;
      for (int n = 0; u0 + 4 * n < u1 && ok; ++n) {
        const int u = u0 + 4 * n + (lane >> 3), i = lane & 7;
        long long k_at = -1, v_at = -1;
        uint8_t ks = 0, vs = 0;
        Segment sg = {};
        if (u < u1) {
          sg = segment_at<ConvertPlan>(p, tab, u, u1);
          const int j = (sg.b0 << 7) + 16 * i;
          if (j < sg.k.len) {
            const int blk = j / p.c.page_size, slot = j - blk * p.c.page_size;
            const int page = page_for_read(p.c, sg.s, blk);
            k_at = page * p.c.k_st[0] + slot * p.c.k_st[1] + sg.h * p.c.k_st[2];
            v_at = page * p.c.v_st[0] + slot * p.c.v_st[1] + sg.h * p.c.v_st[2];
            const long long x = (static_cast<long long>(page) * p.c.hkv + sg.h) * fp.f.per + (slot >> 4);
            ks = fp.f.ks[x];
            vs = fp.f.vs[x];
          }
        }
        const int slot = n % kBatches;
        const bool got = wait_few(u_empty(slot), ((n / kBatches) & 1) ^ 1u, flag, p);
        ok = !__any_sync(0xffffffffu, !got);
        if (!ok) break;
        Unit& to = found[4 * slot + (lane >> 3)];
        to.k_at[i] = k_at;
        to.v_at[i] = v_at;
        to.k_scale[i] = power_of(scale_byte(ks));
        to.v_scale[i] = power_of(scale_byte(vs));
        if (i == 0) {
          to.cached = cached_in(sg.k, sg.b0);
          to.off = sg.k.off;
          to.fresh = sg.b0 == sg.k.db ? sg.k.n : 0;
          to.q0 = sg.k.q0;
          to.h = sg.h;
        }
        warp_arrive(u_full(slot), lane);
      }
    }
  } else if (warp >= L::kConverter0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kConverter));
    // ========================================================= converters
    // A lane has 16 codes of a row, a step of eight warps 32 rows (d = 64: 64; sixteen warps twice that).
    constexpr int kRuns = D / 16, kStep = 32 * L::kConverters / kRuns, kSteps = 128 / kStep;
    const int tid = threadIdx.x - 32 * L::kConverter0, run = tid % kRuns, row0 = tid / kRuns;
    // Where the lane's run of the i-th step lies.  (For two tiles of d = 128 the row's distance is worked out
    // again each time, which is cheaper than the spills that four more registers cost: 64 tokens over 64
    // sequences 342 us instead of 352; elsewhere nothing spills for them, 64 rows 240 instead of 258.)
    auto codes_at = [&](int i, const Unit& un, bool v) -> const uint4* {
      int r = row0;
      if (D == 128 && MT == 2) asm volatile("" : "+r"(r));
      return reinterpret_cast<const uint4*>((v ? fp.f.v : fp.f.k) + (v ? un.v_at : un.k_at)[(r >> 4) + i * kStep / 16] +
                                            (r & 15) * (v ? p.c.v_st[1] : p.c.k_st[1]) + 16 * run);
    };
    // Where the two runs of 8 bf16 elements go (rows of a step further on lie as far on); lanes
    // that would meet in a bank write them in the other order.
    const int half = run >> 2, first = ((2 * run & 7) + half) ^ (row0 & 7);
    uint8_t* const first_at = smem + half * 16384 + (first << 4);
    uint8_t* const second_at = smem + half * 16384 + ((first ^ 1) << 4);
    auto put = [&](uint32_t tile, int row, const uint4& lo, const uint4& hi) {
      *reinterpret_cast<uint4*>(first_at + tile + row * 128) = half ? hi : lo;
      *reinterpret_cast<uint4*>(second_at + tile + row * 128) = half ? lo : hi;
    };
    // K's codes, then V's in their places as K's are converted, then the next block's K's.  (V's in
    // registers of their own, asked for earlier, cost spills: 64 rows 308 us instead of 240.)
    uint4 x[kSteps];
    auto load = [&](int i, const Unit& un, bool v) { x[i] = __ldcs(codes_at(i, un, v)); };
    const int units_here = u1 - u0;
    bool ok = !(p.test_flags & 1u);
    // Unit g's entry; the first of a batch waits for it.
    auto unit = [&](int g) -> const Unit& { return found[g % (4 * kBatches)]; };
    auto arrived = [&](int g) -> bool {
      if ((g & 3) != 0) return true;
      const bool got = wait_bar(u_full(g / 4 % kBatches), (g / 4 / kBatches) & 1, wc);
      return !__any_sync(0xffffffffu, !got);
    };
    ok = ok && arrived(0);
    if (ok && unit(0).cached == 128)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) load(i, unit(0), false);
    for (int g = 0; g < units_here && ok; ++g) {
      const Unit& un = unit(g);
      const int st = g % L::kStages, ph = (g / L::kStages) & 1;
      const int cached = un.cached, off = un.off, fresh = un.fresh;
      const bool more = g + 1 < units_here;
      if (more) ok = arrived(g + 1);
      if (!ok) break;
      const Unit& after = unit(more ? g + 1 : g);
      const bool after_full = more && after.cached == 128;
      // The unit's K or V; what comes next (its V, the next one's K) is asked for as places get free.
      auto convert = [&](uint32_t tile, bool v) {
        const Unit& next = v ? after : un;
        const bool next_full = v ? after_full : cached == 128;
        const float* const scale = (v ? un.v_scale : un.k_scale) + (row0 >> 4);
        if (cached == 128) {
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            uint4 lo, hi;
            to_bf16(x[i], scale[i * kStep / 16], lo, hi);
            put(tile, i * kStep + row0, lo, hi);
            if (next_full) load(i, next, !v);
          }
          return;
        }
        // A tail, new tokens, or both: few of all units, so their codes are read here and the code is short.
        const long long* const fst = v ? fp.vn_st : fp.kn_st;
#pragma unroll 1
        for (int i = 0; i < kSteps; ++i) {
          const int row = i * kStep + row0;
          uint4 lo, hi;
          if (row < cached) {
            to_bf16(*codes_at(i, un, v), scale[i * kStep / 16], lo, hi);
          } else if (row >= off && row < off + fresh) {
            const uint4* const own = reinterpret_cast<const uint4*>((v ? fp.vn : fp.kn) + (un.q0 + row - off) * fst[0] +
                                                                    un.h * fst[1] + 16 * run);
            lo = own[0];
            hi = own[1];
          } else {
            // No key: S is masked there, but a NaN times P's 0 would spread from V.
            if (!v) continue;
            lo = hi = make_uint4(0u, 0u, 0u, 0u);
          }
          put(tile, row, lo, hi);
        }
        if (next_full)
#pragma unroll
          for (int i = 0; i < kSteps; ++i) load(i, next, !v);
      };
      bool got = wait_bar(k_empty(st), ph ^ 1u, wc);
      ok = !__any_sync(0xffffffffu, !got);
      if (!ok) break;
      convert(L::kK + st * L::kTile, false);
      fence_proxy_async_smem();
      warp_arrive(k_full(st), lane);
      got = wait_bar(v_empty(st), ph ^ 1u, wc);
      ok = !__any_sync(0xffffffffu, !got);
      if (!ok) break;
      convert(L::kV + st * L::kTile, true);
      fence_proxy_async_smem();
      warp_arrive(v_full(st), lane);
      // The batch's last entry has been read.
      if ((g & 3) == 3) warp_arrive(u_empty(g / 4 % kBatches), lane);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmax));
    // ============================================================ softmax
    const int tile = MT == 1 ? 0 : (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t t_base = tmem + 256 * tile + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tO = t_base + L::kColO;
    const float sc = p.scale_log2;
    const uint64_t sc2 = pack2(sc, sc);
    int g = 0;  // blocks of this tile
    bool ok = true;
    for (int u = u0; u < u1 && ok;) {
      const Segment sg = segment_at<ConvertPlan>(p, tab, u, u1);
      const bool first_of_cta = u == u0;
      u += sg.b1 - sg.b0;
      const int t0 = sg.m * p.ntt + tile * p.nt, n_rows = min(sg.k.n - t0, p.nt) * p.c.group;
      if (MT == 2 && n_rows <= 0) continue;
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
      // Half x of a block's keys.
      auto block = [&](int b, int x, auto mask_tag) -> bool {
        constexpr bool MASK = decltype(mask_tag)::value;
        const uint32_t tS = t_base + 64 * x;
        const bool got = wait_bar_cold(s_full(tile, x), g & 1, wc);
        if (__any_sync(0xffffffffu, !got)) return false;
        tc_fence_after();
        uint32_t vis[2];
        if constexpr (MASK) {
          const int cv = cached_in(sg.k, b), dn = b == sg.k.db ? sg.k.n : 0;
          const int sh = sg.k.off >> 5, bit = sg.k.off & 31;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
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
        }
        if (active) {
          uint32_t a[32], c2[32];
          float mx = -INFINITY;
          if constexpr (MASK) {
            tmem_ld32(tS, a);
            tmem_ld32(tS + 32, c2);
            tmem_wait_ld();
            reg_fence32(a);
            reg_fence32(c2);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if ((vis[0] >> i) & 1u) mx = fmaxf(mx, __uint_as_float(a[i]));
              if ((vis[1] >> i) & 1u) mx = fmaxf(mx, __uint_as_float(c2[i]));
            }
          } else {
            float m0, m1;
            tmem_ld32_max(tS, a, m0);
            tmem_ld32_max(tS + 32, c2, m1);
            tmem_wait_ld();
            asm volatile("" : "+f"(m0), "+f"(m1));
            reg_fence32(a);
            reg_fence32(c2);
            mx = fmaxf(m0, m1);
          }
          mx *= sc;
          const bool need = r < n_rows && (mx > m_run + kTau || (m_run == -INFINITY && mx > -INFINITY));
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = need ? mx : m_run;
            if (b > sg.b0 || x > 0) {
              const float alpha = need ? ex2_mufu(m_run - m_new) : 1.f;
              // (the product before this one: the other half's, or the last block's)
              const bool landed = wait_bar(pv_done(tile, x ^ 1), (x > 0 ? g : g - 1) & 1, wc);
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
              l_run *= alpha;
            }
            m_run = m_new;
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
            tmem_st16(tS + 16 * c, pk);
          };
          chunk(0, a);
          chunk(1, c2);
          float a0, a1;
          unpack2(fadd2(acc[0], acc[1]), a0, a1);
          l_run += a0 + a1;
          tmem_wait_st();
        }
        tc_fence_before();
        warp_arrive(p_full(tile, x), lane);
        return true;
      };
      for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g)
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x)
          ok = b < sg.k.nfull ? block(b, x, std::false_type{}) : block(b, x, std::true_type{});
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (active) {
        const bool landed = wait_bar_cold(pv_done(tile, 1), (g - 1) & 1, wc);
        if (__any_sync(0xffffffffu, !landed)) { ok = false; break; }
        tc_fence_after();
        const bool whole = sg.b0 == 0 && sg.b1 == sg.k.db + 1;
        const int grp = p.c.group, t = t0 + r / grp, hq = sg.h * grp + r % grp, H = p.c.hkv * grp;
        const long long token = sg.k.q0 + t;
        const int slot = 2 * cta + (first_of_cta ? 0 : 1);
        const int in_part = tile * p.nt * grp + r;
        const long long part = static_cast<long long>(slot) * p.rows + in_part;
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
                auto two = [&](int y) {
                  return pack_bf16x2(__uint_as_float(o8[y]) * inv, __uint_as_float(o8[y + 1]) * inv);
                };
                dst[i] = make_uint4(two(0), two(2), two(4), two(6));
              }
            } else {
              // Row by row, or (many rows) four values of every row side by side.
              const bool wide = p.wide;
              uint4* dst = reinterpret_cast<uint4*>(p.ws_o) +
                           (wide ? (static_cast<long long>(slot) * (D / 4) + 8 * c) * p.rows + in_part : part * (D / 4) + 8 * c);
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
cudaError_t launch(const CacheAttnFp8Launch& a) {
  using L = WL<D, MT>;
  const CacheAttnFp8WideParams p = {a.p, a.f, a.kn, a.vn, {a.kn_st[0], a.kn_st[1]}, {a.vn_st[0], a.vn_st[1]}};
  const unsigned int smem = L::kBytes + 4u * (p.a.c.n_seq + 1);
  static volatile int state[64] = {};  // per device: 0 not checked, 1 usable, -1 not usable
  if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
  if (state[a.device] == 0) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, cache_attn_fp8_wide_kernel<D, MT>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs == Regs<MT>::kLaunch)
      e = cudaFuncSetAttribute(cache_attn_fp8_wide_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               L::kBytes + 4 * (kCacheMaxSeq + 1));
    if (e != cudaSuccess) return e;
    state[a.device] = fa.numRegs == Regs<MT>::kLaunch ? 1 : -1;
  }
  // (the roles' registers would not add up to what the block has, and a role would wait for ever)
  if (state[a.device] < 0) return cudaErrorNotSupported;
  cache_attn_fp8_wide_kernel<D, MT><<<a.grid, L::kThreads, smem, a.stream>>>(a.q_map, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<D, ConvertPlan>(p.a, a.grid, a.stream);
}

}  // namespace

cudaError_t launch_cache_attn_fp8_wide(const CacheAttnFp8Launch& a) {
  if (a.p.c.d == 64) return a.tiles == 2 ? launch<64, 2>(a) : launch<64, 1>(a);
  return a.tiles == 2 ? launch<128, 2>(a) : launch<128, 1>(a);
}

}  // namespace attn
