// The attention weight that each cached key received:
//
//   out_j = in_j + Σ_i Σ_g exp(scale·q_ig·k_j − LSE_ig)
//
// over the query rows i that see key j and the query heads g of its head.  The
// scores are computed with the keys as the M dimension (TMEM lanes), so a thread
// owns one key and sums over the columns: no exchange between threads, no
// atomics, a fixed order.  With few rows the operator is bound by reading k from
// device memory (2d bytes a key), for whole prompts by the exponentials (one per
// 2d flops).
//
// A tile is 256 keys of one (sequence, key head): two M = 128 products per chunk
// of up to 128 query rows, so that each chunk, read from L2, serves 256 keys.  A
// persistent CTA per SM takes the tiles in a fixed order: a sequence's early
// tiles, which most rows see, first, and every second round of CTAs in reverse,
// so that the heaviest tiles and the lightest go to the same CTA.
//
// Where there are few tiles for the SMs (a prompt of 1000 tokens, 8 key heads: 32), a
// cluster of 2, 4 or 8 CTAs takes a tile together (SHARED): each has a run of the tile's
// chunks, and the first adds the others' sums, written into its shared memory, in order.
// Whole prompts, 8 key heads, group 4, d = 128, one CTA a tile and then 2, 4, 8 (us):
// 1000 tokens 32, 21, 15, 18; 2500 tokens 70, 41, 34, 43; 5000 tokens 133, 85, 95, 122;
// 8000 tokens 210, 202, 213, 275; 4000 tokens, 2 key heads, group 8 206, 111, 60, 44.
// (Each CTA loads the tile's keys, and clusters of 8 leave SMs without work.)
//   On the diagonal a warp skips the groups of 32 columns that none of its keys is seen
// by: its chunks have a CTA of their own in a cluster, which the others would wait for.
//
// The −LSE of a column comes out of the tensor core with the score: one more step
// of 16 along the product's inner dimension multiplies a constant (1, 1, 1, 0, …) on
// the keys' side with (hi, mid, lo, 0, …) on the rows', three bf16 numbers that add
// up to −LSE/scale to 24 bits (an infinite hi stands alone).  The sums then read no
// shared memory, whose bandwidth the MMAs' operands fill: with the LSE loaded from there,
// one value for every four bytes of operands, the sums of a chunk took 2.3 times as long
// as the exponentials.
//
// Warps: 0 loads keys; 1 and 2 issue the MMAs of a half each; 3 loads the chunks of
// rows and prepares their columns, a chunk's LSE fetched under the one before; 4-7
// and 8-11 sum a half each, a thread a key: it takes all of a chunk's scores into
// registers at once and gives the S buffer back, so that the tensor core works on the
// next two chunks while the exponentials of one run (twice as many sum warps that
// kept S in TMEM meanwhile took 257 us on a prompt of 8000 tokens, 32 heads over 8 at d = 128,
// where these took 214; now 205).
// TMEM: S of half w, buffer i at columns 256·i + 128·w.  Shared memory holds a ring
// of 128-key slots for each half and one of chunks; a chunk of few rows takes little
// room, which the key rings get (more bytes in flight where memory is the bound).
//   A half has a ring of its own because its issuer has to see every use of a slot: a
// wait on a barrier's parity is only right for the phase after the last one seen.
#include "attn_fwd_kernel.cuh"
#include "cache_device.cuh"

namespace attn {
namespace {

constexpr int kThreadsCW = 384;
constexpr int kTileKeys = 256;

constexpr int kMaxHalf = 4;    // key slots of a half
constexpr int kMaxChunks = 4;  // slots of the chunk ring

template <int D>
struct WL {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kSlot = 128u * D * 2;   // 128 keys: [half][128 rows][128 B]
  static constexpr uint32_t kOnes = 0;              // the keys' side of the added step, 4 KB
  static constexpr int kNumBars = 4 * kMaxHalf + 2 * kMaxChunks + 27;
  static constexpr uint32_t kBar = kOnes + 4096;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;
  static constexpr uint32_t kSums = kMisc + 8;
  static constexpr uint32_t kTable = (kSums + 80 + 15) & ~15u;
  // then the table of n_seq + 1 ints, three ints a sequence, and from a 1024-byte
  // boundary the key rings, the chunks, the rows' sides of their added steps and the
  // other CTAs' sums of a tile
  __host__ __device__ static uint32_t rings(int n_seq) { return (kTable + 4u * (4 * n_seq + 1) + 1023u) & ~1023u; }
};

// Shared-memory matrix descriptor of the added step's operands, without swizzle:
// [two halves of 8 along K][groups of 8 rows][8 rows][16 bytes], the halves 16 bytes a
// row and the groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_added(uint32_t saddr, int rows) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(rows) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// The address in CTA `rank` of the cluster of what is at `saddr` here.
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_in_cluster(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
// Every thread of the cluster's CTAs comes here.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A ring's next slot and the parity of its use (a division by the run-time number of
// slots costs an issuing thread as much as three MMAs).
struct Ring {
  int slots, at = 0;
  uint32_t use = 0;
  __device__ __forceinline__ void next() {
    if (++at == slots) {
      at = 0;
      use ^= 1u;
    }
  }
};

struct WTile {
  int s, h, j0;       // keys [j0, j0 + 256) of sequence s, head h
  int q0, n, rows, len;  // its query rows: first packed row, all of them, those within max_new
  int c0, c1;         // chunks that see a key of the tile: this CTA's share of them
  bool seen;          // whether there are any
};

// `rank`: in the cluster of 2^log_split CTAs that share the tile.  `from`: a sequence
// known to begin at or before tile u (the last one asked for).
__device__ __forceinline__ WTile tile_at(const CacheWeightParams& p, const int* tab, int u, int rank, int log_split, int from = 0) {
  WTile t;
  t.s = u < tab[from + 1] ? from : find_seq(tab, p.c.n_seq, u, from);
  const int* const seq = tab + p.c.n_seq + 1 + 3 * t.s;  // its first row, rows and length
  t.q0 = seq[0];
  t.n = seq[1];
  t.rows = min(t.n, p.c.max_new);
  t.len = seq[2];
  const int rem = u - tab[t.s], kt = p.by_hkv(rem);
  t.h = rem - kt * p.c.hkv;
  t.j0 = kt * kTileKeys;
  // Row i sees slots up to len − n + i: the first that sees slot j0.
  const int first = max(0, t.j0 - t.len + t.n);
  t.c0 = p.by_nt(first);
  t.c1 = max(t.c0, p.by_nt(t.rows + p.nt - 1));
  t.seen = t.c0 < t.c1;
  if (log_split > 0) {
    const int begin = t.c0;
    const long long all = t.c1 - t.c0;
    t.c0 = begin + static_cast<int>(all * rank >> log_split);
    t.c1 = begin + static_cast<int>(all * (rank + 1) >> log_split);
  }
  return t;
}

// The n-th tile of a CTA (or cluster), or -1: rounds of `grid` tiles, every second in
// reverse.
__device__ __forceinline__ int tile_of(int n, int cta, int grid, int units) {
  const long long u = static_cast<long long>(n) * grid + ((n & 1) ? grid - 1 - cta : cta);
  return u < units ? static_cast<int>(u) : -1;
}

// SHARED: clusters share the tiles.
template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreadsCW, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const CacheWeightParams p) {
  using L = WL<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
  auto k_full = [&](int w, int s) { return bars + 8u * (kMaxHalf * w + s); };  // half w, slot s
  auto k_empty = [&](int w, int s) { return bars + 8u * (2 * kMaxHalf + kMaxHalf * w + s); };
  auto q_full = [&](int s) { return bars + 8u * (4 * kMaxHalf + s); };
  auto q_empty = [&](int s) { return bars + 8u * (4 * kMaxHalf + kMaxChunks + s); };
  constexpr uint32_t kB = 4 * kMaxHalf + 2 * kMaxChunks;
  auto s_full = [&](int w, int i) { return bars + 8u * (kB + 2 * w + i); };
  auto s_free = [&](int w, int i) { return bars + 8u * (kB + 4 + 2 * w + i); };
  auto done = [&](int w) { return bars + 8u * (kB + 8 + w); };
  // Of sum warp i: in the first CTA, the others' sums of its keys are there; in the
  // others, the first has taken them.
  auto part_full = [&](int i) { return bars + 8u * (kB + 10 + i); };
  auto part_free = [&](int i) { return bars + 8u * (kB + 18 + i); };
  const uint32_t q_own = bars + 8u * (kB + 26);  // a chunk of which the rows warp zeroes rows
  const int kst = p.k_stages, qst = p.q_stages;  // key slots of a half, chunks
  const uint32_t q_half = static_cast<uint32_t>(p.n_cols) * 128u, q_bytes = q_half * L::kHalves;
  const uint32_t c_bytes = static_cast<uint32_t>(p.n_cols) * 32u;
  const uint32_t ring_k = base + L::rings(p.c.n_seq), ring_q = ring_k + 2 * kst * L::kSlot;
  const uint32_t ring_c = ring_q + qst * q_bytes;
  const uint32_t parts = ring_c + qst * c_bytes;  // [others][256]
  auto k_slot = [&](int w, int s) { return ring_k + (w * kst + s) * L::kSlot; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 4);
  int* const tab = reinterpret_cast<int*>(smem + L::kTable);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (threadIdx.x == 32) {
    *abort_flag = 0u;
    for (int i = 0; i < kMaxHalf; ++i)
      for (int w = 0; w < 2; ++w) {
        mbar_init(k_full(w, i), 1);
        mbar_init(k_empty(w, i), 1);
      }
    for (int i = 0; i < kMaxChunks; ++i) {
      mbar_init(q_full(i), 2);   // its rows, its columns
      mbar_init(q_empty(i), 2);  // both issuers
    }
    for (int w = 0; w < 2; ++w) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(s_full(w, i), 1);
        mbar_init(s_free(w, i), 4);
      }
      mbar_init(done(w), 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(part_full(i), SHARED ? (1 << p.log_split) - 1 : 1);
      mbar_init(part_free(i), 1);
    }
    mbar_init(q_own, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  // The added step's constant side, and zeros where the other side stays zero.
  for (int i = threadIdx.x; i < 256; i += kThreadsCW)
    *reinterpret_cast<uint4*>(smem + L::kOnes + 16 * i) =
        i < 128 ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < 2 * qst * p.n_cols; i += kThreadsCW)
    *reinterpret_cast<uint4*>(smem + (ring_c - base) + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums), [&](int s) {
    const SeqRows r = seq_rows(p.c, s);
    const int len = seq_len(p.c, s);
    int* const seq = tab + p.c.n_seq + 1 + 3 * s;
    seq[0] = r.q0;
    seq[1] = r.n;
    seq[2] = len;
    return p.c.hkv * ((len + kTileKeys - 1) / kTileKeys);
  });
  if constexpr (SHARED) cluster_sync();  // (the barriers are ready for the other CTAs)
  tc_fence_after();
  const int units = tab[p.c.n_seq];
  // Tiles are dealt out to clusters, `cta` of `grid`; more tiles than p.share_most to single CTAs.
  const int log_split = SHARED && units <= p.share_most ? p.log_split : 0, split = 1 << log_split;
  const int rank = blockIdx.x & (split - 1), cta = blockIdx.x >> log_split, grid = gridDim.x >> log_split;
  if (tile_of(0, cta, grid, units) < 0) {
    if (warp == 0) tmem_dealloc(*tmem_slot, 512);
    return;
  }
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  const int nt = p.nt, grp = p.c.group;

  if (warp == 0) {
    // ============================================================= loader
    const int ps = p.piece;
    int filled[2] = {0, 0};   // slots of each half
    Ring rk[2] = {{kst}, {kst}};
    bool ok = true;
    // Lane 8w + i copies the i-th piece of half w, lane 8w waits for its slot; the
    // pages are looked up three tiles ahead, in turn into three sets of registers
    // (moving one set's load results to the next would wait for them: a tile of few
    // rows then took as long as its look-up).
    const int half = lane >> 3, my_row = 128 * half + (lane & 7) * ps;
    auto locate = [&](const WTile& t, int& page, int& slot) {
      const int j = t.j0 + my_row;
      if (lane < 16 && (lane & 7) * ps < 128 && j < t.len) {
        const int blk = p.by_page(j);
        slot = j - blk * p.c.page_size;
        page = page_for_read(p.c, t.s, blk);
      }
    };
    WTile t[3];
    int page[3] = {}, slot[3] = {};
    bool there[3];
    auto fetch = [&](int i, int n, int from) {
      const int u = tile_of(n, cta, grid, units);
      there[i] = u >= 0;
      if (there[i]) {
        t[i] = tile_at(p, tab, u, rank, log_split, from);
        locate(t[i], page[i], slot[i]);
      }
    };
    auto copy = [&](const WTile& t, int page, int slot) {
      const int keys = min(kTileKeys, t.len - t.j0), halves = keys > 128 ? 2 : 1;
      const int npc = half < halves ? (min(128, keys - 128 * half) + ps - 1) / ps : 0;
      const Ring mine_of = half == 1 ? rk[1] : rk[0];
      int mine = 1;
      if ((lane & 7) == 0 && half < halves) {
        mine = wait_bar(k_empty(half, mine_of.at), mine_of.use ^ 1u, wc) && !(p.test_flags & 1u);
        if (mine) mbar_arrive_expect_tx(k_full(half, mine_of.at), static_cast<uint32_t>(npc * ps) * 128u * L::kHalves);
      }
      // A half whose wait ran out is not announced, so nothing of it is copied.
      const unsigned int got = __ballot_sync(0xffffffffu, mine);
      if (half < 2 && (lane & 7) < npc && ((got >> (8 * half)) & 1u))
        for (int hf = 0; hf < L::kHalves; ++hf)
          tma_load_4d(k_slot(half, mine_of.at) + (lane & 7) * ps * 128 + hf * 16384, &tm_k, 64 * hf, t.h, slot, page,
                      k_full(half, mine_of.at));
      __syncwarp();
      ok = got == 0xffffffffu;
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (w < halves && ((got >> (8 * w)) & 1u)) {
          ++filled[w];
          rk[w].next();
        }
    };
    int from = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      fetch(i, i, from);
      if (there[i]) from = t[i].s;
    }
    bool more = true;
    for (int n = 3; ok && more; n += 3) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (!ok || !there[i]) {
          more = false;
          break;
        }
        if (t[i].c0 != t[i].c1) copy(t[i], page[i], slot[i]);  // else no row sees it: nothing to multiply
        fetch(i, n + i, from);
        if (there[i]) from = t[i].s;
      }
    }
    if (lane == 0) {  // no copy may be in flight when the CTA ends, even if only another warp's wait ran out
      const uint64_t t0 = globaltimer_ns();
      auto drain = [&](uint32_t bar, uint32_t parity) {
        while (!mbar_try_wait(bar, parity))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
      };
      for (int w = 0; w < 2; ++w)
        for (int n = max(0, filled[w] - kst); n < filled[w]; ++n) drain(k_full(w, n % kst), (n / kst) & 1u);
    }
  } else if (warp == 1 || warp == 2) {
    // ======================================================== MMA issuers
    if (lane == 0) {
      const uint32_t id = idesc_bf16(128, p.n_cols, false);
      const int w = warp - 1;
      int nq = 0, from = 0;
      Ring rk{kst}, rq{qst};
      bool ok = true;
      for (int n = 0, u; ok && (u = tile_of(n, cta, grid, units)) >= 0; ++n) {
        const WTile t = tile_at(p, tab, u, rank, log_split, from);
        from = t.s;
        if (t.c0 == t.c1) continue;
        // A tile's second half may have no keys: its issuer only keeps count.
        const int halves = t.len - t.j0 > 128 ? 2 : 1;
        const int ks = rk.at;
        if (w < halves) ok = wait_bar(k_full(w, ks), rk.use, wc);
        const uint64_t dk = sdesc_kmajor_sw128(k_slot(w, ks));
        for (int c = t.c0; c < t.c1 && ok; ++c, ++nq, rq.next()) {
          const int qs = rq.at, buf = nq & 1;
          const uint32_t tS = tmem + 256 * buf + 128 * w;
          ok = wait_bar(q_full(qs), rq.use, wc) && wait_bar(s_free(w, buf), ((nq >> 1) & 1) ^ 1u, wc);
          if (!ok) break;
          if (w < halves) {
            tc_fence_after();
            mma_ss(tS, sdesc_added(base + L::kOnes, 128), sdesc_added(ring_c + qs * c_bytes, p.n_cols), id, 0u);
            const uint64_t dq = sdesc_kmajor_sw128(ring_q + qs * q_bytes);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tS, dk + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                     dq + (((kk >> 2) * q_half + (kk & 3) * 32) >> 4), id, 1u);
          }
          mma_commit(s_full(w, buf));
          mma_commit(q_empty(qs));
        }
        if (w < halves) {
          if (ok) mma_commit(k_empty(w, ks));
          rk.next();
        }
      }
      mma_commit(done(w));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(done(w), 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
  } else if (warp == 3) {
    // ================================================================ rows
    // Each chunk's rows, and for each column −LSE/scale (−inf: it adds nothing);
    // lane l has columns l, l + 32, …
    //   A row with an infinite LSE may hold anything in q, and −inf + NaN would be added: such
    // a row is zeroed in shared memory before the chunk is announced.  (Bits of these columns
    // for the sum warps cost every chunk: 215 instead of 204 us on the prompt of 8000.)
    int tk[4];
    const float* src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = lane + 32 * i;
      tk[i] = col < nt * grp ? col / grp : 1 << 30;
      src[i] = p.lse + static_cast<long long>(col % grp) * p.c.total;
    }
    // The chunk after (n, t, c) of this CTA; false at the end.
    int n = 0, u = tile_of(0, cta, grid, units);
    WTile t = tile_at(p, tab, u, rank, log_split);
    int c = t.c0 - 1;
    auto advance = [&]() -> bool {
      ++c;
      while (c >= t.c1) {
        u = tile_of(++n, cta, grid, units);
        if (u < 0) return false;
        t = tile_at(p, tab, u, rank, log_split, t.s);
        c = t.c0;
      }
      return true;
    };
    float v[4];
    auto fetch = [&]() {
      const long long row0 = static_cast<long long>(t.h) * grp * p.c.total + t.q0;
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (nothing of a column without a row is added)
        v[i] = tk[i] < t.rows - c * nt ? src[i][row0 + c * nt + tk[i]] : 0.f;
    };
    bool more = advance();
    if (more) fetch();
    int nq = 0, own = 0;  // chunks; those with rows to zero
    Ring rq{qst};
    for (; more; ++nq, rq.next()) {
      const int qs = rq.at;
      int go = 1;
      if (lane == 0) go = wait_bar(q_empty(qs), rq.use ^ 1u, wc);
      if (!__shfl_sync(0xffffffffu, go, 0)) break;
      bool none = false;  // a row with an infinite LSE
#pragma unroll
      for (int i = 0; i < 4; ++i) none = none || fabsf(v[i]) == INFINITY;
      none = __any_sync(0xffffffffu, none);
      if (lane == 0) {
        const uint32_t bar = none ? q_own : q_full(qs);
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(nt * grp) * 128u * L::kHalves);
        for (int hf = 0; hf < L::kHalves; ++hf)
          tma_load_4d(ring_q + qs * q_bytes + hf * q_half, &tm_q, 64 * hf, 0, t.h, t.q0 + c * nt, bar);
      }
      if (none) {
        const bool landed = wait_bar(q_own, own++ & 1, wc);
        if (__any_sync(0xffffffffu, !landed)) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (fabsf(v[i]) == INFINITY)
            for (int j = 0; j < 8 * L::kHalves; ++j)  // the row's 128 bytes of each half of d
              *reinterpret_cast<uint4*>(smem + (ring_q - base) + qs * q_bytes + (j >> 3) * q_half + (lane + 32 * i) * 128 +
                                        (j & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = v[i] == -INFINITY ? -INFINITY : -v[i] * p.inv_scale;
      more = advance();
      if (more) fetch();
      uint8_t* const col = smem + (ring_c - base) + qs * c_bytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // x = hi + mid + lo, each a rounding to bf16 of what the ones before leave.
        const uint32_t hi = pack_bf16x2(x[i], 0.f) & 0xffffu;
        float rest = x[i] - __uint_as_float(hi << 16);
        if ((hi & 0x7FFFu) == 0x7F80u) rest = 0.f;  // hi = ±inf
        const uint32_t mid = pack_bf16x2(rest, 0.f) & 0xffffu;
        const uint32_t lo = pack_bf16x2(rest - __uint_as_float(mid << 16), 0.f) & 0xffffu;
        if (lane + 32 * i < p.n_cols)
          *reinterpret_cast<uint4*>(col + 16 * (lane + 32 * i)) = make_uint4(hi | (mid << 16), lo, 0u, 0u);
      }
      fence_proxy_async_smem();
      warp_arrive(q_full(qs), lane);
      if (none && lane == 0) mbar_arrive(q_full(qs));  // in place of the copy
    }
    if (lane == 0) {  // no copy may be in flight when the CTA ends, even if only another warp's wait ran out
      const uint64_t t0 = globaltimer_ns();
      for (int i = max(0, nq - qst); i < nq; ++i)
        while (!mbar_try_wait(q_full(i % qst), (i / qst) & 1u))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
      if (own > 0)
        while (!mbar_try_wait(q_own, (own - 1) & 1))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
  } else {
    // =============================================================== sums
    const int w = (warp - 4) >> 2;                     // half of the tile
    const int row = 128 * w + (warp & 3) * 32 + lane;  // key of the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2);
    // The weight gathered so far by this thread's key of tile t: where it is, and
    // the load, issued a tile ahead (under a full memory pipe it takes as long as a
    // tile of few rows; shared tiles have many, and registers are short there).
    auto fetch = [&](const WTile& t, long long& at, float& start) {
      const int key = t.j0 + row;
      at = -1;
      start = 0.f;
      if (key < t.len) {
        const int blk = p.by_page(key);
        const int page = p.c.table[static_cast<long long>(t.s) * p.c.max_blocks + blk];
        if (page >= 0 && page < p.c.n_pages) {
          at = (static_cast<long long>(page) * p.c.hkv + t.h) * p.c.page_size + (key - blk * p.c.page_size);
          if (p.c.weights != nullptr) start = p.c.weights[at];
        }
      }
    };
    int nq = 0, given = 0;  // chunks; tiles whose sums went from CTA to CTA
    bool ok = true;
    int u = tile_of(0, cta, grid, units);
    WTile t = tile_at(p, tab, u, rank, log_split), t_next = t;
    long long at = -1, at_next = -1;
    float start = 0.f, start_next = 0.f;
    if constexpr (!SHARED) fetch(t, at, start);
    for (int n = 0; u >= 0; ++n, t = t_next, at = at_next, start = start_next) {
      u = tile_of(n + 1, cta, grid, units);
      if constexpr (!SHARED) {
        if (u >= 0) {
          t_next = tile_at(p, tab, u, rank, log_split, t.s);
          fetch(t_next, at_next, start_next);
        }
      }
      const int key = t.j0 + row;
      const bool live = t.j0 + 128 * w + (warp & 3) * 32 < t.len;  // this warp has a key
      float total = 0.f;
      for (int c = t.c0; c < t.c1; ++c, ++nq) {
        const int buf = nq & 1, tok0 = c * nt, valid = min(nt, t.rows - tok0) * grp;
        // No mask where the chunk's first row sees the last key of this half.
        const bool masked = min(t.j0 + 128 * w + 127, t.len - 1) > t.len - t.n + tok0;
        const bool got = wait_bar_cold(s_full(w, buf), (nq >> 1) & 1, wc);
        if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tS = tmem + 256 * buf + 128 * w + lane_off;
        uint32_t x[128];
        auto load = [&](int i) { tmem_ld32(tS + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * i])); };
        auto loaded = [&](int i) { reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&x[32 * i])); };
        uint64_t acc[2] = {0, 0};
        // 2^(scale·log2 e·(s − LSE/scale)) over 32 columns.
        auto sum_all = [&](int i0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            unpack2(fmul2(pack2(__uint_as_float(x[i0 + 2 * i]), __uint_as_float(x[i0 + 2 * i + 1])), sc2), a, b);
            acc[i & 1] = fadd2(acc[i & 1], pack2(ex2_mufu(a), ex2_mufu(b)));
          }
        };
        if (live && valid == 128 && !masked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) load(i);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) loaded(i);
          tc_fence_before();
          warp_arrive(s_free(w, buf), lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum_all(32 * i);
        } else {
          if (live) {
            // Columns without a row may hold anything: nothing of them is added.
            // Column i belongs to row tok0 + i / group, which sees slots up to
            // len − n + its number; so the first column that sees this key is
            const int first = masked ? max(0, min(key - (t.len - t.n) - tok0, 128)) * grp : 0;
#pragma unroll 1
            for (int cc = 0; cc < valid; cc += 32) {
              const int from = min(max(first - cc, 0), 32), to = min(valid - cc, 32);
              const uint32_t sees = (from == 32 ? 0u : ~0u << from) & (to == 32 ? ~0u : (1u << to) - 1u);
              if (!__any_sync(0xffffffffu, sees != 0u)) continue;
              tmem_ld32(tS + cc, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
              tmem_wait_ld();
              loaded(0);
              if (__all_sync(0xffffffffu, sees == ~0u)) {
                sum_all(0);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float a, b;
                  unpack2(fmul2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc2), a, b);
                  a = ex2_mufu(a);
                  b = ex2_mufu(b);
                  acc[i & 1] = fadd2(acc[i & 1], pack2((sees >> (2 * i)) & 1u ? a : 0.f, (sees >> (2 * i + 1)) & 1u ? b : 0.f));
                }
              }
            }
          }
          tc_fence_before();
          warp_arrive(s_free(w, buf), lane);
        }
        float a0, a1;
        unpack2(fadd2(acc[0], acc[1]), a0, a1);
        total += a0 + a1;
      }
      if (!ok) break;
      if constexpr (SHARED) {
        if (rank == 0) fetch(t, at, start);
        if (u >= 0) t_next = tile_at(p, tab, u, rank, log_split, t.s);
      }
      if (SHARED && split > 1 && t.seen && live) {
        const int i = warp - 4;
        if (rank > 0) {
          if (given > 0 && __any_sync(0xffffffffu, !wait_bar_cold(part_free(i), (given - 1) & 1, wc))) break;
          fence_cluster();
          store_in_cluster(in_cta(parts + 4u * (256 * (rank - 1) + row), 0), total);
          fence_cluster();
          __syncwarp();
          if (lane == 0) arrive_in_cluster(in_cta(part_full(i), 0));
        } else {
          if (__any_sync(0xffffffffu, !wait_bar_cold(part_full(i), given & 1, wc))) break;
          fence_cluster();
          for (int r = 1; r < split; ++r)
            total += *reinterpret_cast<volatile float*>(smem + (parts - base) + 4 * (256 * (r - 1) + row));
          fence_cluster();
          __syncwarp();
          if (lane > 0 && lane < split) arrive_in_cluster(in_cta(part_free(i), lane));
        }
        ++given;
      }
      if (at >= 0) p.out[at] = start + total;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if constexpr (SHARED) cluster_sync();  // no CTA ends while another may write into it
}

constexpr uint32_t kSmemMax = 232448;

// Clusters of 2^log CTAs that run at a time (they do not cross the GPU's processor
// clusters, so larger ones leave some SMs without work), with all the shared memory that a
// CTA may have; 0 where none does or the runtime does not say.
template <int D>
int clusters_at_a_time(int device, int log, cudaLaunchConfig_t cfg) {
  static volatile int known[64][4] = {};
  int n = known[device][log];
  if (n == 0) {
    cfg.dynamicSmemBytes = kSmemMax;
    if (cudaOccupancyMaxActiveClusters(&n, cache_weights_kernel<D, true>, &cfg) != cudaSuccess) {
      cudaGetLastError();  // (it would be taken for a later launch's)
      return 0;
    }
    known[device][log] = n;
  }
  return n;
}

template <int D, bool SHARED>
cudaError_t launch(const CacheWeightLaunch& a) {
  CacheWeightParams p = a.p;
  if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
  static volatile bool configured[64] = {};
  if (!configured[a.device]) {
    const cudaError_t e =
        cudaFuncSetAttribute(cache_weights_kernel<D, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    configured[a.device] = true;
  }
  // Up to four chunks in flight, and the keys get the rest: a slot for each half (one
  // tile) at least.
  const uint32_t room = kSmemMax - 1024u - WL<D>::rings(p.c.n_seq) - ((1u << p.log_split) - 1u) * 1024u;
  const uint32_t chunk = static_cast<uint32_t>(p.n_cols) * (D * 2 + 32);
  p.q_stages = kMaxChunks;
  while (room - p.q_stages * chunk < 2 * WL<D>::kSlot) --p.q_stages;  // many sequences: their table takes room
  const uint32_t k_stages = (room - p.q_stages * chunk) / (2 * WL<D>::kSlot);
  p.k_stages = static_cast<int>(k_stages < kMaxHalf ? k_stages : kMaxHalf);
  const uint32_t smem = kSmemMax - room + 2 * p.k_stages * WL<D>::kSlot + p.q_stages * chunk;
  if constexpr (!SHARED) {
    cache_weights_kernel<D, false><<<a.grid, kThreadsCW, smem, a.stream>>>(a.q, a.k, p);
    return cudaGetLastError();
  } else {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << p.log_split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1u << p.log_split);
    cfg.blockDim = dim3(kThreadsCW);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int n = clusters_at_a_time<D>(a.device, p.log_split, cfg);
    if (n < 1) {  // each CTA takes whole tiles
      CacheWeightLaunch alone = a;
      alone.p.log_split = 0;
      return launch<D, false>(alone);
    }
    cfg.gridDim.x = static_cast<unsigned int>(n < a.tiles ? n : a.tiles) << p.log_split;
    return cudaLaunchKernelEx(&cfg, cache_weights_kernel<D, true>, a.q, a.k, p);
  }
}

}  // namespace

cudaError_t launch_cache_weights(const CacheWeightLaunch& a) {
  if (a.p.c.d == 64) return a.p.log_split > 0 ? launch<64, true>(a) : launch<64, false>(a);
  return a.p.log_split > 0 ? launch<128, true>(a) : launch<128, false>(a);
}

}  // namespace attn
