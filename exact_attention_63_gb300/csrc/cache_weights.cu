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
// Warps: 0 loads, 1 issues the MMAs, 4-7 and 8-11 sum the two halves of the tile.
// TMEM: S of half w, buffer i at columns 256·i + 128·w.
#include "attn_fwd_kernel.cuh"
#include "cache_device.cuh"

namespace attn {
namespace {

constexpr int kThreadsCW = 384;
constexpr int kTileKeys = 256;

template <int D>
struct WL {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kK1 = 128u * D * 2;               // 128 keys: [half][128 rows][128 B]
  static constexpr int kKStages = 2, kQStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kK = 0, kQ = kKStages * 2 * kK1, kCol = kQ + kQStages * kK1;
  static constexpr uint32_t kBar = kCol + 8 * 128 * 8;        // 8 warps' own copies of (−LSE·log2 e, limit) per column
  static constexpr int kNumBars = 2 * kKStages + 2 * kQStages + 4 + 1;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;
  static constexpr uint32_t kSums = kMisc + 8;
  static constexpr uint32_t kTable = (kSums + 48 + 15) & ~15u;
  static constexpr uint32_t kBytes = kTable + 1024;
};

struct WTile {
  int s, h, j0;       // keys [j0, j0 + 256) of sequence s, head h
  int q0, n, rows, len;  // its query rows: first packed row, all of them, those within max_new
  int c0, c1;         // chunks that see a key of the tile
};

__device__ __forceinline__ int tiles_of(const CacheParams& c, int s) {
  return c.hkv * ((seq_len(c, s) + kTileKeys - 1) / kTileKeys);
}
__device__ __forceinline__ WTile tile_at(const CacheWeightParams& p, const int* tab, int u) {
  WTile t;
  t.s = find_seq(tab, p.c.n_seq, u);
  const SeqRows r = seq_rows(p.c, t.s);
  t.q0 = r.q0;
  t.n = r.n;
  t.rows = min(r.n, p.c.max_new);
  t.len = seq_len(p.c, t.s);
  const int rem = u - tab[t.s];
  t.h = rem % p.c.hkv;
  t.j0 = rem / p.c.hkv * kTileKeys;
  // Row i sees slots up to len − n + i: the first that sees slot j0.
  const int first = max(0, t.j0 - t.len + t.n);
  t.c0 = first / p.nt;
  t.c1 = (t.rows + p.nt - 1) / p.nt;
  t.c1 = max(t.c0, t.c1);
  return t;
}

// The n-th tile of a CTA, or -1: rounds of `grid` tiles, every second in reverse.
__device__ __forceinline__ int tile_of(int n, int cta, int grid, int units) {
  const long long u = static_cast<long long>(n) * grid + ((n & 1) ? grid - 1 - cta : cta);
  return u < units ? static_cast<int>(u) : -1;
}

template <int D>
__global__ void __launch_bounds__(kThreadsCW, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const CacheWeightParams p) {
  using L = WL<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
  auto k_full = [&](int s) { return bars + 8u * s; };
  auto k_empty = [&](int s) { return bars + 8u * (L::kKStages + s); };
  auto q_full = [&](int s) { return bars + 8u * (2 * L::kKStages + s); };
  auto q_empty = [&](int s) { return bars + 8u * (2 * L::kKStages + L::kQStages + s); };
  constexpr uint32_t kB = 2 * L::kKStages + 2 * L::kQStages;
  auto s_full = [&](int i) { return bars + 8u * (kB + i); };
  auto s_free = [&](int i) { return bars + 8u * (kB + 2 + i); };
  const uint32_t done = bars + 8u * (kB + 4);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 4);
  int* const tab = reinterpret_cast<int*>(smem + L::kTable);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, grid = gridDim.x;

  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums), [&](int s) { return tiles_of(p.c, s); });
  const int units = tab[p.c.n_seq];
  if (tile_of(0, cta, grid, units) < 0) return;

  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (threadIdx.x == 32) {
    *abort_flag = 0u;
    for (int i = 0; i < L::kKStages; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_empty(i), 1);
    }
    for (int i = 0; i < L::kQStages; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_free(i), 8);
    }
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};
  const int nt = p.nt, grp = p.c.group;

  if (warp == 0) {
    // ============================================================= loader
    auto waited = [&](uint32_t bar, uint32_t parity) -> bool {
      int ok = 1;
      if (lane == 0) ok = wait_bar(bar, parity, wc);
      return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };
    const int ps = p.piece;
    int nk = 0, nq = 0;
    bool ok = true;
    for (int n = 0, u; ok && (u = tile_of(n, cta, grid, units)) >= 0; ++n) {
      const WTile t = tile_at(p, tab, u);
      if (t.c0 == t.c1) continue;  // no row sees it: nothing to multiply
      // The tile's keys in pieces of ps rows: lane i has the i-th.
      const int keys = min(kTileKeys, t.len - t.j0), npc = (keys + ps - 1) / ps;
      int page = 0, slot = 0;
      if (lane < npc) {
        const int j = t.j0 + lane * ps, blk = j / p.c.page_size;
        slot = j - blk * p.c.page_size;
        page = page_for_read(p.c, t.s, blk);
      }
      const int ks = nk % L::kKStages;
      ok = waited(k_empty(ks), ((nk / L::kKStages) & 1) ^ 1u);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(k_full(ks), static_cast<uint32_t>(npc * ps) * 128u * L::kHalves);
      __syncwarp();
      if (lane < npc) {
        const int row = lane * ps;
        const uint32_t dst = base + L::kK + (2 * ks + (row >> 7)) * L::kK1 + (row & 127) * 128;
        for (int hf = 0; hf < L::kHalves; ++hf) tma_load_4d(dst + hf * 16384, &tm_k, 64 * hf, t.h, slot, page, k_full(ks));
      }
      __syncwarp();
      ++nk;
      for (int c = t.c0; c < t.c1 && ok; ++c) {
        const int qs = nq % L::kQStages;
        ok = waited(q_empty(qs), ((nq / L::kQStages) & 1) ^ 1u);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full(qs), static_cast<uint32_t>(nt * grp) * 128u * L::kHalves);
          for (int hf = 0; hf < L::kHalves; ++hf)
            tma_load_4d(base + L::kQ + qs * L::kK1 + hf * 16384, &tm_q, 64 * hf, 0, t.h, t.q0 + c * nt, q_full(qs));
        }
        ++nq;
      }
    }
    if (lane == 0 && !ok) {  // no copy may be in flight when the CTA ends
      const uint64_t t0 = globaltimer_ns();
      auto drain = [&](uint32_t bar, uint32_t parity) {
        while (!mbar_try_wait(bar, parity))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
      };
      for (int n = max(0, nk - L::kKStages); n < nk; ++n) drain(k_full(n % L::kKStages), (n / L::kKStages) & 1u);
      for (int n = max(0, nq - L::kQStages); n < nq; ++n) drain(q_full(n % L::kQStages), (n / L::kQStages) & 1u);
    }
  } else if (warp == 1) {
    // ========================================================= MMA issuer
    if (lane == 0) {
      const uint32_t id = idesc_bf16(128, p.n_cols, false);
      int nk = 0, nq = 0;
      bool ok = true;
      for (int n = 0, u; ok && (u = tile_of(n, cta, grid, units)) >= 0; ++n) {
        const WTile t = tile_at(p, tab, u);
        if (t.c0 == t.c1) continue;
        const int ks = nk % L::kKStages;
        ok = wait_bar(k_full(ks), (nk / L::kKStages) & 1, wc);
        for (int c = t.c0; c < t.c1 && ok; ++c, ++nq) {
          const int qs = nq % L::kQStages, buf = nq & 1;
          ok = wait_bar(q_full(qs), (nq / L::kQStages) & 1, wc) && wait_bar(s_free(buf), ((nq >> 1) & 1) ^ 1u, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dq = sdesc_kmajor_sw128(base + L::kQ + qs * L::kK1);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint64_t dk = sdesc_kmajor_sw128(base + L::kK + (2 * ks + w) * L::kK1);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
              mma_ss(tmem + 256 * buf + 128 * w, dk + o, dq + o, id, kk > 0 ? 1u : 0u);
            }
          }
          mma_commit(s_full(buf));
          mma_commit(q_empty(qs));
          if (c == t.c1 - 1) mma_commit(k_empty(ks));
        }
        ++nk;
      }
      mma_commit(done);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(done, 0))
        if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
  } else if (warp >= 4) {
    // =============================================================== sums
    const int w = (warp - 4) >> 2;                       // half of the tile
    const int row = 128 * w + (warp & 3) * 32 + lane;    // key of the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* const col_lse = reinterpret_cast<float*>(smem + L::kCol) + (warp - 4) * 256;
    int* const col_lim = reinterpret_cast<int*>(col_lse + 128);
    const uint64_t sc2 = pack2(p.scale_log2, p.scale_log2);
    int nq = 0;
    bool ok = true;
    for (int n = 0, u; ok && (u = tile_of(n, cta, grid, units)) >= 0; ++n) {
      const WTile t = tile_at(p, tab, u);
      const int key = t.j0 + row;
      float total = 0.f;
      for (int c = t.c0; c < t.c1; ++c, ++nq) {
        const int buf = nq & 1;
        const int tok0 = c * nt;
        // This warp's copy of the columns' −LSE·log2 e (−inf: adds nothing) and
        // of the last slot each one sees.
        __syncwarp();
        for (int col = lane; col < 128; col += 32) {
          const int tk = tok0 + col / grp, g = col - (col / grp) * grp;
          float v = -INFINITY;
          if (col < nt * grp && tk < t.rows) {
            v = -p.lse[static_cast<long long>(t.h * grp + g) * p.c.total + t.q0 + tk] * 1.4426950408889634f;
            if (v == INFINITY) v = -INFINITY;
          }
          col_lse[col] = v;
          col_lim[col] = t.len - t.n + tk;
        }
        __syncwarp();
        const bool got = wait_bar_cold(s_full(buf), (nq >> 1) & 1, wc);
        if (__any_sync(0xffffffffu, !got)) { ok = false; break; }
        tc_fence_after();
        // No mask where the chunk's first row sees the last key of this half.
        const bool masked = min(t.j0 + 128 * w + 127, t.len - 1) > t.len - t.n + tok0;
        float sum = 0.f;
        for (int cc = 0; cc < p.n_cols; cc += 32) {
          uint32_t x[32];
          tmem_ld32(tmem + 256 * buf + 128 * w + cc + lane_off, x);
          tmem_wait_ld();
          reg_fence32(x);
          uint64_t acc[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 nl = *reinterpret_cast<const float2*>(&col_lse[cc + 2 * i]);
            float a, b;
            unpack2(ffma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc2, pack2(nl.x, nl.y)), a, b);
            a = ex2_mufu(a);
            b = ex2_mufu(b);
            // A column without a row may hold anything.
            if (nl.x == -INFINITY) a = 0.f;
            if (nl.y == -INFINITY) b = 0.f;
            if (masked) {
              if (key > col_lim[cc + 2 * i]) a = 0.f;
              if (key > col_lim[cc + 2 * i + 1]) b = 0.f;
            }
            acc[i & 1] = fadd2(acc[i & 1], pack2(a, b));
          }
          float a0, a1;
          unpack2(fadd2(acc[0], acc[1]), a0, a1);
          sum += a0 + a1;
        }
        total += sum;
        tc_fence_before();
        warp_arrive(s_free(buf), lane);
      }
      if (!ok) break;
      if (key < t.len) {
        const int blk = key / p.c.page_size;
        const int page = p.c.table[static_cast<long long>(t.s) * p.c.max_blocks + blk];
        if (page >= 0 && page < p.c.n_pages) {
          const long long at = (static_cast<long long>(page) * p.c.hkv + t.h) * p.c.page_size + (key - blk * p.c.page_size);
          p.out[at] = (p.c.weights != nullptr ? p.c.weights[at] : 0.f) + total;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const CacheWeightLaunch& a) {
  const unsigned int smem = WL<D>::kBytes + 4u * (a.p.c.n_seq + 1);
  static volatile bool configured[64] = {};
  if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
  if (!configured[a.device]) {
    const cudaError_t e = cudaFuncSetAttribute(cache_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               WL<D>::kBytes + 4 * (kCacheMaxSeq + 1));
    if (e != cudaSuccess) return e;
    configured[a.device] = true;
  }
  cache_weights_kernel<D><<<a.grid, kThreadsCW, smem, a.stream>>>(a.q, a.k, a.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_weights(const CacheWeightLaunch& a) { return a.p.c.d == 64 ? launch<64>(a) : launch<128>(a); }

}  // namespace attn
