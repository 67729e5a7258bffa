// The cache's bookkeeping operators: appending rows, choosing the tokens that
// stay, moving them together.  All three are bound by memory (append, compact)
// or by the passes over a head's weights in shared memory (select).
#include "attn_gb300.h"
#include "cache_device.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------- append
// One warp copies one token's k or v: H_kv·d·2 bytes, 16 a lane, four loads in
// flight.  The k warps also set the weights and positions.
__global__ void __launch_bounds__(256) cache_append_kernel(const CacheAppendParams p) {
  const CacheParams& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long wi = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int i = static_cast<int>(wi >> 1), which = static_cast<int>(wi & 1);
  if (i >= p.n_rows) return;
  // The last sequence s with cu[s] <= i, 32 candidates a step.
  int lo = 0, n = c.n_seq;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = lane * step < n && c.cu[at] <= i;
    const unsigned int votes = __ballot_sync(0xffffffffu, le);
    const int k = votes == 0u ? 0 : 31 - __clz(votes);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int a = min(max(c.cu[lo], 0), p.n_rows), z = min(max(c.cu[lo + 1], a), p.n_rows);
  if (i < a || i >= z) return;
  const int len = seq_len(c, lo), slot = len - z + i;
  if (slot < 0) return;
  const int src = p.rows != nullptr ? p.rows[i] : i;
  if (src < 0 || src >= c.total) return;
  const int blk = slot / c.page_size, js = slot - blk * c.page_size;
  const int page = c.table[static_cast<long long>(lo) * c.max_blocks + blk];
  if (page < 0 || page >= c.n_pages) return;

  const long long* const st = which ? c.v_st : c.k_st;
  const long long* const ns = which ? p.vn_st : p.kn_st;
  uint16_t* const dst = (which ? c.v : c.k) + page * st[0] + js * st[1];
  const uint16_t* const from = (which ? p.vn : p.kn) + src * ns[0];
  const int sh = c.d == 128 ? 4 : 3, chunks = c.hkv << sh, mask = (1 << sh) - 1;
  for (int q = lane; q < chunks; q += 128) {
    uint4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int qq = q + 32 * e;
      if (qq < chunks) x[e] = *reinterpret_cast<const uint4*>(from + (qq >> sh) * ns[1] + (qq & mask) * 8);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int qq = q + 32 * e;
      if (qq < chunks) *reinterpret_cast<uint4*>(dst + (qq >> sh) * st[2] + (qq & mask) * 8) = x[e];
    }
  }
  if (which == 0) {
    const int pos = (p.seq_pos != nullptr ? p.seq_pos[lo] : len) - z + i;
    for (int h = lane; h < c.hkv; h += 32) {
      const long long at = (static_cast<long long>(page) * c.hkv + h) * c.page_size + js;
      if (c.weights != nullptr) c.weights[at] = 0.f;
      if (c.positions != nullptr) c.positions[at] = pos;
    }
  }
}

// ------------------------------------------------------------------ compact
// One warp looks at 32 entries of kept and moves the rows of those beyond the
// budget: d/8 lanes of 16 bytes a row, k and v side by side, four rows in flight.
__global__ void __launch_bounds__(256) cache_compact_kernel(const CacheParams c, const int* kept, int budget) {
  const int lane = threadIdx.x & 31;
  const long long wi = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int tiles = (budget + 31) / 32;
  const long long sh = wi / tiles;
  const int s = static_cast<int>(sh / c.hkv), h = static_cast<int>(sh % c.hkv);
  if (s >= c.n_seq) return;
  const int i = static_cast<int>(wi % tiles) * 32 + lane;
  int from = -1;
  if (i < budget) from = kept[sh * budget + i];
  bool move = from >= budget && from < c.cap && i < c.cap;
  long long k0 = 0, k1 = 0, v0 = 0, v1 = 0;
  if (move) {
    const int* const tab = c.table + static_cast<long long>(s) * c.max_blocks;
    const int b0 = from / c.page_size, j0 = from - b0 * c.page_size, b1 = i / c.page_size, j1 = i - b1 * c.page_size;
    const int p0 = tab[b0], p1 = tab[b1];
    move = p0 >= 0 && p0 < c.n_pages && p1 >= 0 && p1 < c.n_pages;
    if (move) {
      k0 = p0 * c.k_st[0] + j0 * c.k_st[1];
      k1 = p1 * c.k_st[0] + j1 * c.k_st[1];
      v0 = p0 * c.v_st[0] + j0 * c.v_st[1];
      v1 = p1 * c.v_st[0] + j1 * c.v_st[1];
      const long long a0 = (static_cast<long long>(p0) * c.hkv + h) * c.page_size + j0;
      const long long a1 = (static_cast<long long>(p1) * c.hkv + h) * c.page_size + j1;
      if (c.weights != nullptr) c.weights[a1] = c.weights[a0];
      if (c.positions != nullptr) c.positions[a1] = c.positions[a0];
    }
  }
  unsigned int todo = __ballot_sync(0xffffffffu, move);
  const int per = c.d / 8, grp = lane / per, at = (lane % per) * 8, both = 32 / per / 2;  // rows a step: 1 or 2
  const bool is_v = grp & 1;
  const uint16_t* const src = (is_v ? c.v + h * c.v_st[2] : c.k + h * c.k_st[2]) + at;
  uint16_t* const dst = (is_v ? c.v + h * c.v_st[2] : c.k + h * c.k_st[2]) + at;
  while (todo) {
    uint4 x[4];
    long long to[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // This lane's row: the (grp/2)-th of the next `both` entries.
      int mine = -1;
      for (int b = 0; b < both; ++b) {
        const int j = todo ? __ffs(todo) - 1 : -1;
        todo &= todo - 1;  // 0 stays 0
        if (b == (grp >> 1)) mine = j;
      }
      const int l = max(mine, 0);
      const long long fk = __shfl_sync(0xffffffffu, k0, l), fv = __shfl_sync(0xffffffffu, v0, l);
      const long long tk = __shfl_sync(0xffffffffu, k1, l), tv = __shfl_sync(0xffffffffu, v1, l);
      to[e] = mine < 0 ? -1 : (is_v ? tv : tk);
      if (mine >= 0) x[e] = *reinterpret_cast<const uint4*>(src + (is_v ? fv : fk));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (to[e] >= 0) *reinterpret_cast<uint4*>(dst + to[e]) = x[e];
  }
}

// ------------------------------------------------------------------- select
// One CTA ranks one (sequence, head).  The budget-th largest key is found digit
// by digit (11, 11 and 10 bits) from histograms in shared memory; one pass then
// marks the slots that stay in a bit map (of those equal to the threshold, the
// first ones), and the k-th freed slot below n takes the k-th kept slot behind it.
// Keys stay in shared memory where a sequence fits, and the kept slots behind n are
// then listed over them; else each pass reads the weights again, and a binary search
// over the map's counts finds the k-th.  Four keys a lane and step: with the loads
// coalesced the passes are bound by their instructions.
constexpr int kThreadsSel = 1024;
constexpr int kBins = 2048;
constexpr uint32_t kSmemMax = 232448;

// Larger key = stays earlier: 0xffffffff for the newest, then the weight in the
// order of its bits, 0 for NaN.
__device__ __forceinline__ uint32_t rank_key(float w, bool newest) {
  if (newest) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);  // −0 as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The map keeps a group of 128 slots as four ballots: bit l of word e is slot 4l + e.
struct Group {
  uint32_t b[4];
  // Set slots in the lanes given by the mask.
  __device__ __forceinline__ int count(uint32_t lanes) const {
    return __popc(b[0] & lanes) + __popc(b[1] & lanes) + __popc(b[2] & lanes) + __popc(b[3] & lanes);
  }
  __device__ __forceinline__ uint32_t nibble(int l) const {
    return ((b[0] >> l) & 1u) | (((b[1] >> l) & 1u) << 1) | (((b[2] >> l) & 1u) << 2) | (((b[3] >> l) & 1u) << 3);
  }
  // The k-th (from 0) set slot.
  __device__ __forceinline__ int nth(int k) const {
    int l = 0;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      const int below = count(((1u << w) - 1u) << l);
      if (k >= below) {
        k -= below;
        l += w;
      }
    }
    uint32_t x = nibble(l);
    for (; k > 0; --k) x &= x - 1;
    return 4 * l + __ffs(x) - 1;
  }
};

struct SelectSmem {
  uint32_t words, groups, keys;  // bit-map words, groups of four words, cached keys
  uint32_t offset;               // of the keys, bytes
};
__host__ __device__ inline SelectSmem select_smem(int cap) {
  SelectSmem m;
  m.groups = static_cast<uint32_t>((cap + 127) / 128);
  m.words = 4 * m.groups;
  m.offset = (kBins * 4 + 64 * 4 + m.words * 4 + m.groups * 4 + 15) & ~15u;
  const uint32_t room = (kSmemMax - m.offset) / 16 * 4;
  m.keys = room < static_cast<uint32_t>(cap) ? room : static_cast<uint32_t>(cap);  // cap: a multiple of 16
  return m;
}
inline uint32_t select_bytes(int cap) {
  const SelectSmem m = select_smem(cap);
  return m.offset + m.keys * 4;
}

// Exclusive sum over the CTA's threads, and the total; `w`: 33 ints.
__device__ __forceinline__ int block_exclusive(int v, int* w, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) w[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int x = w[lane];
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    w[lane] = s - x;
    if (lane == 31) w[32] = s;
  }
  __syncthreads();
  const int r = w[warp] + incl - v;
  *total = w[32];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kThreadsSel)
    cache_select_kernel(const CacheParams c, const int* seq_pos, int budget, int recent, int* kept) {
  extern __shared__ __align__(16) uint32_t sel_smem[];
  const SelectSmem lay = select_smem(c.cap);
  int* const hist = reinterpret_cast<int*>(sel_smem);
  int* const scratch = hist + kBins;  // 33 for scans, then [40] digit, [41] count above
  uint32_t* const bits = reinterpret_cast<uint32_t*>(scratch + 64);
  int* const before = reinterpret_cast<int*>(bits + lay.words);
  uint4* const kq = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(sel_smem) + lay.offset);  // four keys each

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / c.hkv, h = blockIdx.x - s * c.hkv;
  const int len = seq_len(c, s), n = min(len, budget);
  int* const out = kept + static_cast<long long>(blockIdx.x) * budget;
  for (int i = n + tid; i < budget; i += kThreadsSel) out[i] = -1;
  if (len <= budget) {
    for (int i = tid; i < n; i += kThreadsSel) out[i] = i;
    return;
  }
  const int* const tab = c.table + static_cast<long long>(s) * c.max_blocks;
  const long long newest = (c.positions != nullptr ? static_cast<long long>(seq_pos[s]) : len) - recent;
  // Four slots at a time: page_size is a multiple of four, so they share a page.
  // The up to three behind the last slot count as slots with the lowest key: they
  // come last of all, and more than budget others come before.
  const int quads = (len + 3) / 4;
  auto load_quad = [&](int b, int off, int j) -> uint4 {
    const int page = min(max(tab[b], 0), c.n_pages - 1);
    const long long at = (static_cast<long long>(page) * c.hkv + h) * c.page_size + off;
    const float4 w = *reinterpret_cast<const float4*>(c.weights + at);
    int4 pos = make_int4(j, j + 1, j + 2, j + 3);
    if (c.positions != nullptr) pos = *reinterpret_cast<const int4*>(c.positions + at);
    return make_uint4(rank_key(w.x, pos.x >= newest), j + 1 < len ? rank_key(w.y, pos.y >= newest) : 0u,
                      j + 2 < len ? rank_key(w.z, pos.z >= newest) : 0u,
                      j + 3 < len ? rank_key(w.w, pos.w >= newest) : 0u);
  };
  const bool cached = len <= static_cast<int>(lay.keys);
  auto quad_of = [&](int q) -> uint4 {
    if (cached) return kq[q];
    const int b = 4 * q / c.page_size;
    return load_quad(b, 4 * q - b * c.page_size, 4 * q);
  };

  // ---- threshold: the budget-th largest key, and how many equal to it stay
  uint32_t prefix = 0, fixed_bits = 0;
  int want = budget;  // rank of the threshold among the keys that match the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), width = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kThreadsSel) hist[i] = 0;
    __syncthreads();
    const uint32_t digit = (1u << width) - 1u;
    auto count = [&](uint4 k) {
      const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((x[e] & fixed_bits) == prefix) atomicAdd(&hist[(x[e] >> shift) & digit], 1);
    };
    if (pass == 0) {
      const int db = 4 * kThreadsSel / c.page_size, doff = 4 * kThreadsSel - db * c.page_size;
      int b = 4 * tid / c.page_size, off = 4 * tid - b * c.page_size;
      for (int q0 = tid; q0 < quads; q0 += 4 * kThreadsSel) {
        uint4 k[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = q0 + e * kThreadsSel;
          if (q < quads) k[e] = load_quad(b, off, 4 * q);
          b += db;
          off += doff;
          if (off >= c.page_size) {
            off -= c.page_size;
            ++b;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = q0 + e * kThreadsSel;
          if (q < quads) {
            if (cached) kq[q] = k[e];
            count(k[e]);
          }
        }
      }
    } else {
#pragma unroll 4
      for (int q = tid; q < quads; q += kThreadsSel) count(quad_of(q));
    }
    __syncthreads();
    // Bins from the top: thread t has bins kBins − 1 − 2t and the next lower one.
    const int hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
    int total;
    const int above = block_exclusive(hi + lo, scratch, &total);
    if (above < want && want <= above + hi + lo) {
      const bool in_hi = want <= above + hi;
      scratch[40] = kBins - 1 - 2 * tid - (in_hi ? 0 : 1);
      scratch[41] = above + (in_hi ? 0 : hi);
      scratch[42] = in_hi ? hi : lo;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(scratch[40]) << shift;
    fixed_bits |= ((1u << width) - 1u) << shift;
    want -= scratch[41];
    __syncthreads();
  }
  const uint32_t thr = prefix;
  const bool ties = scratch[42] > want;  // more keys equal the threshold than may stay

  // ---- the map of the slots that stay; each warp has a run of groups of 128
  // slots, a lane four of them
  const int groups = (len + 127) / 128, per = (groups + 31) / 32;
  const int g0 = min(groups, warp * per), g1 = min(groups, g0 + per);
  const uint32_t lanes_below = (1u << lane) - 1u;
  auto quad_in = [&](int g) { return g * 32 + lane < quads ? quad_of(g * 32 + lane) : make_uint4(0u, 0u, 0u, 0u); };
  auto four = [](bool x, bool y, bool z, bool w) { return (x ? 1u : 0u) | (y ? 2u : 0u) | (z ? 4u : 0u) | (w ? 8u : 0u); };
  auto ballots = [&](uint32_t nib) -> Group {
    return {{__ballot_sync(0xffffffffu, nib & 1u), __ballot_sync(0xffffffffu, nib & 2u),
             __ballot_sync(0xffffffffu, nib & 4u), __ballot_sync(0xffffffffu, nib & 8u)}};
  };
  auto put = [&](int g, const Group& x) {
    if (lane == 0) reinterpret_cast<uint4*>(bits)[g] = make_uint4(x.b[0], x.b[1], x.b[2], x.b[3]);
  };
  auto get = [&](int g) -> Group {
    const uint4 x = reinterpret_cast<const uint4*>(bits)[g];
    return {{x.x, x.y, x.z, x.w}};
  };
  // Of the nibble of slots 4·lane … of group g: those at or beyond n.
  auto behind = [&](uint32_t nib, int g) {
    const int first = g * 128 + 4 * lane;
    return nib & (0xfu << max(0, min(n - first, 4))) & 0xfu;
  };
  auto behind_of = [&](int g, const Group& x) -> Group {
    return g * 128 >= n ? x : ballots(behind(x.nibble(lane), g));
  };
  int src = 0;  // kept slots at or beyond n in this warp's run
  int total;
  auto count_behind = [&](int g, const Group& x) {
    if (lane == 0) before[g] = src;
    if (g * 128 + 128 > n) src += behind_of(g, x).count(0xffffffffu);
  };
  if (!ties) {
    // (The threshold is not the padding's 0 here: as many keys as may stay equal it.)
    for (int g = g0; g < g1; ++g) {
      const uint4 k = quad_in(g);
      const Group x = ballots(four(k.x >= thr, k.y >= thr, k.z >= thr, k.w >= thr));
      put(g, x);
      count_behind(g, x);
    }
  } else {
    int eq = 0;
    for (int g = g0; g < g1; ++g) {
      const uint4 k = quad_in(g);
      eq += g * 32 + lane < quads ? __popc(four(k.x == thr, k.y == thr, k.z == thr, k.w == thr)) : 0;
    }
    eq = __reduce_add_sync(0xffffffffu, eq);
    int eq_before = block_exclusive(lane == 0 ? eq : 0, scratch, &total);
    eq_before = __shfl_sync(0xffffffffu, eq_before, 0);
    for (int g = g0; g < g1; ++g) {
      const uint4 k = quad_in(g);
      uint32_t nib = four(k.x > thr, k.y > thr, k.z > thr, k.w > thr);
      const uint32_t ne = g * 32 + lane < quads ? four(k.x == thr, k.y == thr, k.z == thr, k.w == thr) : 0u;
      const Group equal = ballots(ne);
      int room = want - eq_before - equal.count(lanes_below);  // of the equal ones the first stay
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((ne >> e) & 1u) {
          if (room > 0) nib |= 1u << e;
          --room;
        }
      eq_before += equal.count(0xffffffffu);
      const Group x = ballots(nib);
      put(g, x);
      count_behind(g, x);
    }
  }
  int src_before = block_exclusive(lane == 0 ? src : 0, scratch, &total);
  src_before = __shfl_sync(0xffffffffu, src_before, 0);
  for (int g = g0 + lane; g < g1; g += 32) before[g] += src_before;
  __syncwarp();

  // ---- the kept slots at or beyond n, listed over the keys
  int* const list = reinterpret_cast<int*>(kq);
  if (cached) {
    for (int g = max(g0, n / 128); g < g1; ++g) {
      const Group x = behind_of(g, get(g));
      const uint32_t nib = x.nibble(lane);
      int at = before[g] + x.count(lanes_below);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((nib >> e) & 1u) list[at++] = g * 128 + 4 * lane + e;
    }
  }
  __syncthreads();

  // ---- slots below n: kept where they are, or filled by the k-th kept slot behind
  const int gn = (n + 127) / 128, gper = (gn + 31) / 32;
  const int h0 = min(gn, warp * gper), h1 = min(gn, h0 + gper);
  auto freed = [&](int g) -> Group {  // the slots below n that do not stay
    const Group x = get(g);
    if (g * 128 + 128 <= n) return {{~x.b[0], ~x.b[1], ~x.b[2], ~x.b[3]}};
    return ballots(~x.nibble(lane) & ~behind(0xfu, g));
  };
  int holes = 0;
  for (int g = h0; g < h1; ++g) holes += freed(g).count(0xffffffffu);
  int hole_before = block_exclusive(lane == 0 ? holes : 0, scratch, &total);
  hole_before = __shfl_sync(0xffffffffu, hole_before, 0);
  for (int g = h0; g < h1; ++g) {
    const Group x = freed(g);
    const uint32_t nib = x.nibble(lane);
    int k = hole_before + x.count(lanes_below);
    hole_before += x.count(0xffffffffu);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = g * 128 + 4 * lane + e;
      int from = j;
      if ((nib >> e) & 1u) {
        if (cached) {
          from = list[k];
        } else {
          int lo = n / 128, hi = groups - 1;  // the last group with before[lo] <= k
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= k) lo = mid;
            else hi = mid - 1;
          }
          // (the group with slot n has kept slots below n too)
          Group y = get(lo);
          const int skip = max(0, n - lo * 128);
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int gone = max(0, min((skip - f + 3) / 4, 32));  // lanes whose slot f is below n
            y.b[f] = gone == 32 ? 0u : y.b[f] & (~0u << gone);
          }
          from = lo * 128 + y.nth(k - before[lo]);
        }
        ++k;
      }
      if (j < n) out[j] = from;
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t stream) {
  const long long warps = 2ll * p.n_rows;
  cache_append_kernel<<<static_cast<unsigned int>((warps + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheParams& c, const int* kept, int budget, cudaStream_t stream) {
  const long long warps = static_cast<long long>(c.n_seq) * c.hkv * ((budget + 31) / 32);
  cache_compact_kernel<<<static_cast<unsigned int>((warps + 7) / 8), 256, 0, stream>>>(c, kept, budget);
  return cudaGetLastError();
}

cudaError_t launch_cache_select(const CacheParams& c, const int* seq_pos, int budget, int recent, int* kept, int device,
                                cudaStream_t stream) {
  static volatile bool configured[64] = {};
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!configured[device]) {
    const cudaError_t e =
        cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    configured[device] = true;
  }
  cache_select_kernel<<<c.n_seq * c.hkv, kThreadsSel, select_bytes(c.cap), stream>>>(c, seq_pos, budget, recent, kept);
  return cudaGetLastError();
}

}  // namespace attn
