// Attention of new tokens over a paged cache of E4M3 codes and over each other, few rows.
//
//   s_tj = scale·q_t·k_j,  O_t = Σ_j exp(s_tj − LSE_t)·v_j,  LSE_t = ln Σ_j exp(s_tj),
// with k_j = 2^a·K_j and v_j = 2^b·V_j for the cached keys (codes K, V; a, b of the block of
// 16 slots and key head), bf16 rows for the new tokens.
//
// The rows of one (sequence, key head) are its (token, head of the group) pairs, eight a
// column tile of the matrix instruction.  With few of them the operator is bound by reading
// the codes: 2d bytes a key.  So everything between memory and the sums is kept short.  The
// M side of the m16n8k16 products is the cache:  Sᵀ = K·Qᵀ (16 keys × 8 rows), Oᵀ += Vᵀ·Pᵀ
// (16 values × 8 rows); which key or element a fragment's row or column stands for is free
// as long as both sides agree, so a lane reads whole runs of 16 bytes of the cache, and a code
// becomes an f16 number (exactly) in one instruction for two.
//   A warp has a key head and every (16 / hg)-th block of 16 slots of its CTA's range, a block
// being one block of scales: 2^a is one factor of its scores, 2^b one of its product, which
// is added to O in fp32.  Each warp copies the bytes that it will read itself, lanes for one
// another (in order by their wait and a __syncwarp before the reads, one after them), so nothing is
// handed from warp to warp: no wait of one for another before the end of a tile, where the warps
// of a head meet.  (With a loading warp and TMA the copies' issue set the pace, two
// to four cycles a row of 128 or 64 bytes: 146 us for one token over 64 sequences of up to
// 8191 at d = 128, 113 at d = 64.)
//   Q's rows are scaled by a power of two to a maximum of 2^14 … 2^15 before they become f16:
// values down to 2^−28 of the largest keep all eight bits, the rest are off by less than
// 2^−39 of it, less than the fp32 sum of the products.  P, in units where the running
// maximum is 2^7 (at most 2^15 until it is moved), is rounded to f16: 2^−11 relative, and
// what lies below f16's range is less than 2^−32 of the largest.  The fp32 sums hold n keys with
// |v| up to 2^113 / n.  The factor of a row's scores is its power of two times the block's 2^a: it leaves
// fp32 at scale·max|q|·2^a = 2^141, and its first part is subnormal below scale·max|q| = 2^−111.
//
// Work units are blocks of 128 / hg keys of hg key heads (8 where the number of heads is a
// multiple of 8) of one sequence and row tile, 32 KB of codes at d = 128, dealt out evenly
// as in cache_attn.cu, a range for each CTA or (up to 8 rows, where tiles are many) for each of its two
// groups of eight warps; the parts of a tile are joined by the same second kernel.  With all
// heads of a token in one block the pages are read as they lie (hg = 1: 220 us where 8 takes
// 146, before the copies).
#include "cache_join.cuh"
#include "fp8_device.cuh"

namespace attn {
namespace {

constexpr float kShift = 7.0f;  // log2 of P where a score is the reference maximum
constexpr float kTau = 8.0f;    // log2: the reference moves when exceeded by more
constexpr float kNone = -3e38f; // the reference before any score
constexpr int kLookUp = 16;     // blocks looked up at a time

struct CacheAttnFp8Params {
  CacheAttnParams a;
  Fp8Pages f;
  const uint16_t* q;
  const uint16_t* kn;
  const uint16_t* vn;
  long long q_st[2], kn_st[2], vn_st[2];
  bool apart;            // a range of units for each group of eight warps instead of each CTA
};

// The blocks of 128 / hg cached keys; the new tokens go with the last.
struct RowsPlan {
  static constexpr bool kEight = true, kRuns = true;
  static constexpr int most_rows(int d) { return d == 128 ? 16 : 32; }
  static __device__ __forceinline__ KeyPlan of(const CacheAttnParams& p, int s) {
    KeyPlan k;
    const SeqRows r = seq_rows(p.c, s);
    k.q0 = r.q0;
    k.n = min(r.n, p.c.max_new);
    k.len = seq_len(p.c, s);
    const int keys = 128 / p.hg;
    k.nfull = k.tail = k.off = 0;  // (of the other kernel's blocks)
    k.db = max((k.len + keys - 1) / keys, 1) - 1;
    return k;
  }
};

// D = A·B + C, m16n8k16.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1,
                                    float c2, float c3) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool add) {
  if (add) mma<F16>(d, a, b0, b1, d[0], d[1], d[2], d[3]);
  else mma<F16>(d, a, b0, b1, 0.f, 0.f, 0.f, 0.f);
}
// Transposes an 8 × 8 tile of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ld_shared_v2(uint32_t addr, uint32_t (&r)[2]) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A block's 16 rows of D bytes in shared memory: where 16-byte run c of row r lies.
template <int D>
__device__ __forceinline__ uint32_t run_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}
// The key that row (of Sᵀ) or column (of Vᵀ) i < 8 of a fragment stands for, i + 8 for the
// key 8 further.  With run_at's places neither the rows 2q and 2q + 1 of K that eight lanes
// read together, nor the columns 2t of V, meet in a bank.
template <int D>
__device__ __forceinline__ int key_of(int i) {
  const int t = i >> 1;
  return D == 128 ? (2 * t + (t >> 1)) ^ ((i & 1) << 2) : i ^ (t & 1);
}

template <int D, int NT>
struct FL {
  static constexpr int kGroups = NT == 1 ? 2 : 1;        // of eight warps: a unit is one group's
  static constexpr int kWarps = 8 * kGroups;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kKeys = 16u * D;             // bytes of a block's K or V, of one head
  static constexpr bool kQShared = NT > 2;               // Q's fragments do not fit beside O
  static constexpr int kStages = (D == 128 ? 3 : 6) * (NT == 2 ? 2 : 1);  // blocks of a warp: one at work, the others on their way
  static_assert(kStages <= kLookUp - 3, "the next blocks' pages are looked up three blocks ahead of them");
  static constexpr uint32_t kRing = 0;                   // [warp][stage][K, V][16 rows]
  static constexpr uint32_t kMergeWarp = NT * D / 32 * 32 * 16;  // half of a warp's O, as its lanes hold it
  static constexpr uint32_t kQ = kWarps * kStages * 2 * kKeys;   // [warp][two products][tile][lane]
  static constexpr uint32_t kMerge = kQ + (kQShared ? kWarps * NT * D / 16 * 256 : 0);
  static constexpr uint32_t kMl = kMerge + 4 * kGroups * kMergeWarp;  // [8][NT][2][lane] maximum and sum
  static constexpr uint32_t kOffsets = kMl + 8 * NT * 2 * 32 * 8;    // [warp][kLookUp] of K and V, bytes
  static constexpr uint32_t kScales = kOffsets + kWarps * kLookUp * 16;  // [warp][stage] bytes of K and V
  static constexpr uint32_t kSums = kScales + kWarps * kStages * 2;
  static constexpr uint32_t kTable = (kSums + 4 * kWarps + 15) & ~15u;
  static constexpr uint32_t kBytes = kTable + 128;       // + alignment; the table comes on top
};

template <int D, int NT>
__global__ void __launch_bounds__(FL<D, NT>::kThreads, 1) cache_attn_fp8_kernel(const CacheAttnFp8Params fp) {
  using L = FL<D, NT>;
  const CacheAttnParams& p = fp.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 127u) & ~127u;
  uint8_t* const smem = smem_raw + (base - raw);
  int* const tab = reinterpret_cast<int*>(smem + L::kTable);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums),
               [&](int s) { return units_of<RowsPlan>(p, s); });
  const int units = tab[p.c.n_seq];
  if (cta == 0)
    for (int i = threadIdx.x; i <= p.c.n_seq; i += L::kThreads) p.ws_table[i] = tab[i];
  // The ranges of units: a CTA's, or (apart) one for each of its two groups of warps.
  const int gr = lane >> 2, t4 = lane & 3, group = warp >> 3, part8 = warp & 7;
  const bool apart = L::kGroups > 1 && fp.apart;
  const int groups = apart ? 1 : L::kGroups, share = apart ? 0 : group;  // that share a range; which of them
  const int range = apart ? cta + group * static_cast<int>(gridDim.x) : cta;
  const int grid = min(static_cast<int>(gridDim.x) * (apart ? 2 : 1), units);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (range >= grid) return;
  const int u0 = range_start(units, range, grid), u1 = range_start(units, range + 1, grid);

  const int hg = p.hg, hh = part8 & (hg - 1), tb = part8 / hg, per_block = 8 / hg, keys = 128 / hg;
  const int grp = p.c.group, H = p.c.hkv * grp;
  constexpr int kSteps = D / 16;  // m16n8k16 products of a score tile, and tiles of Oᵀ

  // ---- the warp's blocks: number x is the tb-th 16 slots of unit u0 + share + groups·x.  16 of
  // them are looked up at a time, a lane each, while earlier ones are worked on: their pages first, and
  // with few registers in use (NT = 1) two blocks later their places and scales, so that
  // neither is waited for (one token over 64 sequences 130 -> 128 us, d = 64 76 -> 74; with
  // more rows the registers make it 3 % slower).
  constexpr bool kTwice = NT == 1;
  struct Page {
    int page, slot, h;     // page −1: nothing to copy
  };
  struct Block {
    long long k, v;        // offsets of its first row; −1: nothing to copy
    uint32_t ks, vs;       // scales
  };
  auto find_page = [&](int x) -> Page {
    Page r = {-1, 0, 0};
    const int u = u0 + share + groups * (x + lane);
    if (u >= u1 || lane >= kLookUp) return r;
    const Segment sg = segment_at<RowsPlan>(p, tab, u, u1);
    const int j = sg.b0 * keys + 16 * tb;
    if (j >= sg.k.len) return r;
    const int blk = j / p.c.page_size;
    r.slot = j - blk * p.c.page_size;
    r.h = sg.h * hg + hh;
    r.page = page_for_read(p.c, sg.s, blk);
    return r;
  };
  auto find_block = [&](const Page& at) -> Block {
    Block r = {-1, -1, 0u, 0u};
    if (at.page < 0) return r;
    r.k = at.page * p.c.k_st[0] + at.slot * p.c.k_st[1] + at.h * p.c.k_st[2];
    r.v = at.page * p.c.v_st[0] + at.slot * p.c.v_st[1] + at.h * p.c.v_st[2];
    const long long i = (static_cast<long long>(at.page) * p.c.hkv + at.h) * fp.f.per + (at.slot >> 4);
    r.ks = fp.f.ks[i];
    r.vs = fp.f.vs[i];
    return r;
  };
  // The warp's places in shared memory: where this lane copies to (its row of the first 4 or 8,
  // 16 bytes), and the rows and runs of the fragments that it reads.
  const uint32_t ring = base + L::kRing + warp * L::kStages * 2 * L::kKeys;
  constexpr int kRunsRow = D / 16, kRowsStep = 32 / kRunsRow, kSteps16 = 16 / kRowsStep;  // runs a row; rows a copy
  const int my_row = lane / kRunsRow, my_run = lane % kRunsRow;
  const uint32_t to[2] = {ring + run_at<D>(my_row, my_run), ring + run_at<D>(my_row + kRowsStep, my_run)};
  uint32_t k_at[2][D / 64], v_at[2];
#pragma unroll
  for (int hf = 0; hf < D / 64; ++hf) {
    k_at[0][hf] = ring + run_at<D>(key_of<D>(gr), 4 * hf + t4);
    k_at[1][hf] = ring + run_at<D>(8 + key_of<D>(gr), 4 * hf + t4);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v_at[i] = ring + L::kKeys + run_at<D>(key_of<D>(2 * t4 + i), D == 128 ? gr : gr >> 1) + (D == 128 ? 0 : 8 * (gr & 1));
  uint16_t* const scales = reinterpret_cast<uint16_t*>(smem + L::kScales) + warp * L::kStages;
  longlong2* const offsets = reinterpret_cast<longlong2*>(smem + L::kOffsets) + warp * kLookUp;
  const uint8_t* const k_lane = fp.f.k + my_row * p.c.k_st[1] + 16 * my_run;
  const uint8_t* const v_lane = fp.f.v + my_row * p.c.v_st[1] + 16 * my_run;
  auto publish = [&](const Block& r) {
    __syncwarp();
    if (lane < kLookUp) offsets[lane] = make_longlong2(r.k, r.v);
    __syncwarp();
  };
  auto copy = [&](int x, int st) {
    const longlong2 off = offsets[x & (kLookUp - 1)];
    if (off.x >= 0) {
      const uint8_t *const k = k_lane + off.x, *const v = v_lane + off.y;
      const uint32_t at = st * 2 * L::kKeys;
#pragma unroll
      for (int i = 0; i < kSteps16; ++i)
        copy_async(to[i & 1] + at + (i >> 1) * 2 * kRowsStep * D, k + i * kRowsStep * p.c.k_st[1]);
#pragma unroll
      for (int i = 0; i < kSteps16; ++i)
        copy_async(to[i & 1] + L::kKeys + at + (i >> 1) * 2 * kRowsStep * D, v + i * kRowsStep * p.c.v_st[1]);
    }
    copy_commit();
  };
  auto keep_scales = [&](const Block& r, int x, int st) {
    if (lane == (x & (kLookUp - 1))) scales[st] = static_cast<uint16_t>(r.ks | r.vs << 8);
  };
  Block now = find_block(find_page(0));
  publish(now);
#pragma unroll 1
  for (int x = 0; x < L::kStages; ++x) copy(x, x);
#pragma unroll 1
  for (int x = 0; x < L::kStages; ++x) keep_scales(now, x, x);
  Page next_at = {-1, 0, 0};
  Block next = {-1, -1, 0u, 0u};
  if (!kTwice) next = find_block(find_page(kLookUp));

  int x = 0, st = 0;  // the block at work and its place in the ring
  for (int u = u0; u < u1;) {
    const Segment sg = segment_at<RowsPlan>(p, tab, u, u1);
    const bool first_of_range = u == u0;
    u += sg.b1 - sg.b0;
    const int h = sg.h * hg + hh, row0 = sg.m * p.rows, n_rows = min(sg.k.n * grp - row0, p.rows);
    // ---- Q: the rows of this thread's fragments (row gr of each tile), as f16
    uint32_t qf[L::kQShared ? 1 : NT][kSteps][2];
    uint4* const q_own = reinterpret_cast<uint4*>(smem + L::kQ) + warp * (NT * kSteps / 2) * 32 + lane;
    float mult[NT][2];  // of the scores in its columns (rows 2·t4 and 2·t4 + 1)
    auto q_row = [&](int r) {
      const int rr = row0 + min(r, n_rows - 1);
      return fp.q + (sg.k.q0 + rr / grp) * fp.q_st[0] + (h * grp + rr % grp) * fp.q_st[1];
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint16_t* const src = q_row(8 * nt + gr);
      uint32_t w[D / 64][8], top = 0u;
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf) {
        const uint4 lo = *reinterpret_cast<const uint4*>(src + 64 * hf + 16 * t4);
        const uint4 hi = *reinterpret_cast<const uint4*>(src + 64 * hf + 16 * t4 + 8);
        w[hf][0] = lo.x; w[hf][1] = lo.y; w[hf][2] = lo.z; w[hf][3] = lo.w;
        w[hf][4] = hi.x; w[hf][5] = hi.y; w[hf][6] = hi.z; w[hf][7] = hi.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, max(w[hf][i] & 0x7FFFu, (w[hf][i] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int up = min(141 - static_cast<int>(top >> 7), 127);  // the row's maximum becomes 2^14 … 2^15
      const float f = power_of(127 + up), inv = p.scale_log2 * power_of(127 - min(up, 126));
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // two products
          uint32_t two[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[hf][4 * j + i];
            two[i] = pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
          }
          if constexpr (L::kQShared) {
            q_own[((2 * hf + j) * NT + nt) * 32] = make_uint4(two[0], two[1], two[2], two[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[nt][4 * hf + 2 * j + i / 2][i & 1] = two[i];
          }
        }
      const float rest = up == 127 ? 0.5f * inv : inv;  // (2^−127 is no normal number)
      mult[nt][0] = __shfl_sync(0xffffffffu, rest, 8 * t4);
      mult[nt][1] = __shfl_sync(0xffffffffu, rest, 8 * t4 + 4);
    }
    // O, sums and references: pairs of columns (rows 2·t4 and 2·t4 + 1 of Q) side by side.
    uint64_t o[NT][kSteps][2], l_run[NT];
    float m_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < kSteps; ++c) o[nt][c][0] = o[nt][c][1] = 0ull;
      m_run[nt][0] = m_run[nt][1] = kNone;
      l_run[nt] = 0ull;
    }
    // Products s of the tile to P, 2^(s·f − reference + 7), 0 where `hidden`.  A reference
    // that is exceeded by more than kTau moves, and with it O and the sums.
    auto weigh = [&](float(&s)[NT][4], const float(&f)[NT][2], auto hidden) {
      float e[NT][4], top = -INFINITY;
      auto exponents = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint64_t f2 = pack2(f[nt][0], f[nt][1]), r2 = pack2(kShift - m_run[nt][0], kShift - m_run[nt][1]);
          unpack2(ffma2(pack2(s[nt][0], s[nt][1]), f2, r2), e[nt][0], e[nt][1]);
          unpack2(ffma2(pack2(s[nt][2], s[nt][3]), f2, r2), e[nt][2], e[nt][3]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (hidden(nt, i)) e[nt][i] = -INFINITY;
        }
      };
      exponents();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top = fmaxf(top, fmaxf(fmaxf(e[nt][0], e[nt][1]), fmaxf(e[nt][2], e[nt][3])));
      if (__any_sync(0xffffffffu, top > kShift + kTau)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float alpha[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = m_run[nt][i];
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (!hidden(nt, i + 2 * y)) m = fmaxf(m, s[nt][i + 2 * y] * f[nt][i]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            alpha[i] = m == m_run[nt][i] ? 1.f : ex2_mufu(m_run[nt][i] - m);
            m_run[nt][i] = m;
          }
          const uint64_t a2 = pack2(alpha[0], alpha[1]);
          l_run[nt] = fmul2(l_run[nt], a2);
#pragma unroll
          for (int c = 0; c < kSteps; ++c) {
            o[nt][c][0] = fmul2(o[nt][c][0], a2);
            o[nt][c][1] = fmul2(o[nt][c][1], a2);
          }
        }
        exponents();
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = ex2_mufu(e[nt][i]);
        l_run[nt] = fadd2(fadd2(l_run[nt], pack2(s[nt][0], s[nt][1])), pack2(s[nt][2], s[nt][3]));
      }
    };
    // One block of 16 keys, `nv` of them of the sequence (all, without MASK).
    auto block = [&](int nv, auto mask_tag) {
      constexpr bool MASK = decltype(mask_tag)::value;
      const uint32_t at = st * 2 * L::kKeys, sc = scales[st];
      uint32_t kw[D / 32][4];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) ld_shared_v4(k_at[i & 1][i >> 1] + at, kw[i]);
      const float ka = power_of(scale_byte(sc & 0xFFu)), vb = power_of(scale_byte(sc >> 8));
      // (two sums a tile: half the chain of products)
      float s[NT][4], s2[L::kQShared ? 1 : NT][4], f[NT][2];
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
          uint4 qq[L::kQShared ? NT : 1];
          if constexpr (L::kQShared)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) qq[nt] = q_own[((2 * hf + j2) * NT + nt) * 32];
#pragma unroll
          for (int j = 2 * j2; j < 2 * j2 + 2; ++j) {
            const uint32_t lo = kw[2 * hf][j], hi = kw[2 * hf + 1][j];
            const uint32_t a[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(lo >> 16),
                                   e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (L::kQShared)
                mma<true>(s[nt], a, j & 1 ? qq[nt].z : qq[nt].x, j & 1 ? qq[nt].w : qq[nt].y, hf > 0 || j > 0);
              else
                mma<true>(j & 1 ? s2[nt] : s[nt], a, qf[nt][4 * hf + j][0], qf[nt][4 * hf + j][1], hf > 0 || j > 1);
            }
          }
        }
      // Keys 2·t4, 2·t4 + 1 and both + 8, this lane's run of D / 8 values.
      uint32_t w[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) ld_shared_v4(v_at[i & 1] + at + (i >> 1) * 8 * D, w[i]);
        else ld_shared_v2(v_at[i & 1] + at + (i >> 1) * 8 * D, w[i]);
        // (codes behind the sequence's end: their P is 0, but a NaN would spread)
        if (MASK && key_of<D>(2 * t4 + (i & 1)) + 4 * (i & 2) >= nv)
#pragma unroll
          for (int y = 0; y < D / 32; ++y) w[i][y] = 0u;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if constexpr (!L::kQShared) s[nt][i] += s2[nt][i];
        f[nt][0] = mult[nt][0] * ka;
        f[nt][1] = mult[nt][1] * ka;
      }
      weigh(s, f, [&](int, int i) { return MASK && key_of<D>(gr) + (i & 2 ? 8 : 0) >= nv; });
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pf[nt][0] = transposed(pack_f16x2(s[nt][0], s[nt][1]));
        pf[nt][1] = transposed(pack_f16x2(s[nt][2], s[nt][3]));
      }
      const uint64_t vb2 = pack2(vb, vb);
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        // Values 2c and 2c + 1 of the run, in pairs of keys.
        const uint32_t w0 = __byte_perm(w[0][c >> 1], w[1][c >> 1], c & 1 ? 0x7362 : 0x5140),
                       w1 = __byte_perm(w[2][c >> 1], w[3][c >> 1], c & 1 ? 0x7362 : 0x5140);
        const uint32_t a[4] = {e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w0 >> 16), e4m3x2_to_f16x2(w1),
                               e4m3x2_to_f16x2(w1 >> 16)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pv[4];
          mma<true>(pv, a, pf[nt][0], pf[nt][1], false);
          o[nt][c][0] = ffma2(pack2(pv[0], pv[1]), vb2, o[nt][c][0]);
          o[nt][c][1] = ffma2(pack2(pv[2], pv[3]), vb2, o[nt][c][1]);
        }
      }
    };

    for (;; ++x) {
      // (units of the segment come in order: its last is u − 1)
      const int unit = u0 + share + groups * x;
      if (unit >= u) break;
      copy_wait<L::kStages - 1>();
      __syncwarp();
      const int nv = sg.k.len - (sg.b1 - (u - unit)) * keys - 16 * tb;  // keys from the block's first on
      if (nv >= 16) block(16, std::false_type{});
      else if (nv > 0) block(nv, std::true_type{});
      // The block's place is free: on with the one that is kStages ahead.
      const int ahead = x + L::kStages;
      const int phase = ahead & (kLookUp - 1);
      if (kTwice && phase == kLookUp - 3) next_at = find_page(ahead + 3);
      if (kTwice && phase == kLookUp - 1) next = find_block(next_at);
      if (phase == 0) {
        now = next;
        publish(now);
        if (!kTwice) next = find_block(find_page(ahead + kLookUp));
      }
      __syncwarp();  // (every lane has read the block: it holds bytes that others copied)
      copy(ahead, st);
      keep_scales(now, ahead, st);
      st = st + 1 == L::kStages ? 0 : st + 1;
    }
    // ---- the new tokens' own keys, 16 at a time, from the head's last warp on (whose cached keys
    // are often none)
    const int sharers = per_block * groups;
#pragma unroll 1
    for (int k0 = 16 * (sharers - 1 - (tb + per_block * share)); sg.b1 == sg.k.db + 1 && k0 < sg.k.n;
         k0 += 16 * sharers) {
      uint32_t mine = 0u;  // which of the 16 keys row `lane` of the tile sees
      {
        const int t = (row0 + min(lane, n_rows - 1)) / grp;
        uint32_t anc[4] = {0u, 0u, 0u, 0u};
        if (p.parents == nullptr) {
          const int n = min(max(t + 1 - k0, 0), 16);
          mine = (1u << n) - 1u;
        } else {
          ancestors(p.parents + sg.k.q0, sg.k.n, t, lane, anc);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i == k0 >> 5) mine = (anc[i] >> (k0 & 16)) & 0xffffu;
        }
      }
      const uint16_t* const kn = fp.kn + static_cast<long long>(h) * fp.kn_st[1];
      const uint16_t* const vn = fp.vn + static_cast<long long>(h) * fp.vn_st[1];
      const int ja = k0 + gr, jb = ja + 8;
      float s[NT][4], f[NT][2];
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int it = 0; it < D / 32; ++it) {
        const int c = (4 * it + t4) * 8;
        const uint4 ka = ja < sg.k.n ? *reinterpret_cast<const uint4*>(kn + (sg.k.q0 + ja) * fp.kn_st[0] + c) : zero;
        const uint4 kb = jb < sg.k.n ? *reinterpret_cast<const uint4*>(kn + (sg.k.q0 + jb) * fp.kn_st[0] + c) : zero;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 q = *reinterpret_cast<const uint4*>(q_row(8 * nt + gr) + c);
          const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
          mma<false>(s[nt], a0, q.x, q.y, it > 0);
          mma<false>(s[nt], a1, q.z, q.w, true);
        }
      }
      uint32_t see[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          see[nt][i] = __shfl_sync(0xffffffffu, mine, 8 * nt + 2 * t4 + i) >> gr;
          f[nt][i] = p.scale_log2;
        }
      weigh(s, f, [&](int nt, int i) { return ((see[nt][i & 1] >> (i & 2 ? 8 : 0)) & 1u) == 0u; });
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pf[nt][0] = transposed(pack_bf16x2(s[nt][0], s[nt][1]));
        pf[nt][1] = transposed(pack_bf16x2(s[nt][2], s[nt][3]));
      }
      uint4 y[4][D / 64];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = k0 + 2 * t4 + (i & 1) + 4 * (i & 2);
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          y[i][e] = j < sg.k.n ? *reinterpret_cast<const uint4*>(vn + (sg.k.q0 + j) * fp.vn_st[0] + D / 8 * gr + 8 * e) : zero;
      }
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        auto word = [&](int i) {
          const uint4& z = y[i][c >> 2];
          return (c & 3) == 0 ? z.x : (c & 3) == 1 ? z.y : (c & 3) == 2 ? z.z : z.w;
        };
        const uint32_t a[4] = {__byte_perm(word(0), word(1), 0x5410), __byte_perm(word(0), word(1), 0x7632),
                               __byte_perm(word(2), word(3), 0x5410), __byte_perm(word(2), word(3), 0x7632)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float z[4];
          unpack2(o[nt][c][0], z[0], z[1]);
          unpack2(o[nt][c][1], z[2], z[3]);
          mma<false>(z, a, pf[nt][0], pf[nt][1], true);
          o[nt][c][0] = pack2(z[0], z[1]);
          o[nt][c][1] = pack2(z[2], z[3]);
        }
      }
    }
    // ---- the warps of a head meet: half of them hand their maxima, sums and O to the other
    // half, until one is left
    // `pair`: by a barrier of the two warps that share the slot, otherwise by one of all warps,
    // since the next level's pairs are others.
    auto all = [&]() {  // warps that go through the same segments
      asm volatile("bar.sync %0, %1;" ::"r"(9 + (apart ? group : 0)), "r"(apart ? 256 : 32 * L::kWarps) : "memory");
    };
    auto meet = [&](int slot, bool gives, bool takes, auto pair) {
      auto both = [&]() {
        if constexpr (decltype(pair)::value) asm volatile("bar.sync %0, 64;" ::"r"(1 + slot) : "memory");
        else all();
      };
      float4* const ml = reinterpret_cast<float4*>(smem + L::kMl) + slot * NT * 32 + lane;
      ulonglong2* const half = reinterpret_cast<ulonglong2*>(smem + L::kMerge + slot * L::kMergeWarp) + lane;
      uint64_t ours[NT], theirs[NT];
      if (gives)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float l0, l1;
          unpack2(l_run[nt], l0, l1);
          ml[nt * 32] = make_float4(m_run[nt][0], m_run[nt][1], l0, l1);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (gives)
#pragma unroll
          for (int i = 0; i < NT * kSteps / 2; ++i) {
            const uint64_t(&y)[2] = o[i / (kSteps / 2)][x * (kSteps / 2) + i % (kSteps / 2)];
            half[i * 32] = make_ulonglong2(y[0], y[1]);
          }
        both();
        if (takes) {
          if (x == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float4 y = ml[nt * 32];
              const float their_m[2] = {y.x, y.y};
              float a[2], b[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float& m = m_run[nt][i];
                const float top = fmaxf(m, their_m[i]);
                // (a warp that saw nothing has sum and O of 0, or NaN that stays)
                a[i] = m == top ? 1.f : ex2_mufu(m - top);
                b[i] = their_m[i] == top ? 1.f : ex2_mufu(their_m[i] - top);
                m = top;
              }
              ours[nt] = pack2(a[0], a[1]);
              theirs[nt] = pack2(b[0], b[1]);
              l_run[nt] = ffma2(pack2(y.z, y.w), theirs[nt], fmul2(l_run[nt], ours[nt]));
            }
#pragma unroll
          for (int i = 0; i < NT * kSteps / 2; ++i) {
            const ulonglong2 y = half[i * 32];
            const int nt = i / (kSteps / 2);
            uint64_t(&z)[2] = o[nt][x * (kSteps / 2) + i % (kSteps / 2)];
            z[0] = ffma2(y.x, theirs[nt], fmul2(z[0], ours[nt]));
            z[1] = ffma2(y.y, theirs[nt], fmul2(z[1], ours[nt]));
          }
        }
        both();
      }
    };
    if (groups > 1) {
      meet(part8, group == 1, group == 0, std::true_type{});  // (warps part8 and part8 + 8)
      if (per_block > 1) all();
    }
    for (int w = per_block / 2; w > 0; w >>= 1)
      meet((apart ? 4 * group : 0) + hh + hg * (tb & (w - 1)), share == 0 && tb >= w && tb < 2 * w, share == 0 && tb < w,
           std::false_type{});
    if (share != 0 || tb != 0) continue;
    // ---- the head's rows, by its one warp
    const bool whole = sg.b0 == 0 && sg.b1 == sg.k.db + 1;
    const int slot = 2 * range + (first_of_range ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l_run[nt] = fadd2(l_run[nt], __shfl_xor_sync(0xffffffffu, l_run[nt], x));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nt + 2 * t4 + i;
        if (r >= n_rows) continue;
        auto of = [&](uint64_t two) {  // this row's of a pair
          float a, b;
          unpack2(two, a, b);
          return i ? b : a;
        };
        const float l = of(l_run[nt]), m = l == 0.f ? -INFINITY : m_run[nt][i] - kShift;
        if (whole) {
          const int rr = row0 + r, hq = h * grp + rr % grp;
          const long long token = sg.k.q0 + rr / grp;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint4* const dst = reinterpret_cast<uint4*>(p.o + (token * H + hq) * D + D / 8 * gr);
#pragma unroll
          for (int e = 0; e < D / 64; ++e) {
            auto two = [&](int c) { return pack_bf16x2(of(o[nt][4 * e + c][0]) * inv, of(o[nt][4 * e + c][1]) * inv); };
            dst[e] = make_uint4(two(0), two(1), two(2), two(3));
          }
          if (gr == 0)
            p.lse[static_cast<long long>(hq) * p.c.total + token] =
                l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
        } else {
          const long long part = (static_cast<long long>(slot) * hg + hh) * p.rows + r;
          float4* const dst = reinterpret_cast<float4*>(p.ws_o + part * D + D / 8 * gr);
#pragma unroll
          for (int e = 0; e < D / 32; ++e)
            dst[e] = make_float4(of(o[nt][2 * e][0]), of(o[nt][2 * e][1]), of(o[nt][2 * e + 1][0]), of(o[nt][2 * e + 1][1]));
          if (gr == 0) p.ws_ml[part] = make_float2(m, l);
        }
      }
    }
  }
}

template <int D, int NT>
cudaError_t launch(const CacheAttnFp8Launch& a) {
  using L = FL<D, NT>;
  CacheAttnFp8Params p = {a.p, a.f, a.q, a.kn, a.vn, {a.q_st[0], a.q_st[1]}, {a.kn_st[0], a.kn_st[1]}, {a.vn_st[0], a.vn_st[1]}, a.apart};
  const unsigned int smem = L::kBytes + 4u * (p.a.c.n_seq + 1);
  static volatile bool configured[64] = {};
  if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
  if (!configured[a.device]) {
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_fp8_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               L::kBytes + 4 * (kCacheMaxSeq + 1));
    if (e != cudaSuccess) return e;
    configured[a.device] = true;
  }
  cache_attn_fp8_kernel<D, NT><<<a.grid, L::kThreads, smem, a.stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<D, RowsPlan>(p.a, a.apart ? 2 * a.grid : a.grid, a.stream);
}

}  // namespace

cudaError_t launch_cache_attn_fp8(const CacheAttnFp8Launch& a) {
  if (a.p.c.d == 64) return a.p.rows > 16 ? launch<64, 4>(a) : a.p.rows > 8 ? launch<64, 2>(a) : launch<64, 1>(a);
  return a.p.rows > 8 ? launch<128, 2>(a) : launch<128, 1>(a);  // (more rows: the other kernel)
}

}  // namespace attn
