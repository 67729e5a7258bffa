// Attention of new tokens over a paged cache of E4M3 codes and over each other.
//
//   s_tj = scale·q_t·k_j,  O_t = Σ_j exp(s_tj − LSE_t)·v_j,  LSE_t = ln Σ_j exp(s_tj),
// with k_j = 2^a·K_j and v_j = 2^b·V_j for the cached keys (codes K, V; a, b of the block of
// 16 slots and key head), bf16 rows for the new tokens.
//
// The rows of one (sequence, key head) are its (token, head of the group) pairs, eight a
// column tile of the matrix instruction.  With few of them the operator is bound by reading
// the codes: 2d bytes a key.  So everything between memory and the sums is kept short: a
// code becomes an f16 number in one instruction for two (its four bits are exact there), and
// goes from the ring straight into the fragments of m16n8k16 products whose M side is the
// cache:  Sᵀ = K·Qᵀ (16 keys × 8 rows), Oᵀ += Vᵀ·Pᵀ (16 values × 8 rows).  Codes taken to
// bf16 tiles in shared memory for tcgen05 would cross it three times more, 6 bytes an
// element where 5.5 are all that its 128 bytes a cycle leave at the copy rate.
//   A warp's 16 keys are one block of scales, so 2^a is one factor of its scores and 2^b one
// of its product, which is added to O in fp32.
//   Q's rows are scaled by a power of two to a maximum of 2^14 … 2^15 before they become f16:
// values down to 2^−28 of the largest keep all eight bits, the rest are off by less than
// 2^−39 of it, less than the fp32 sum of the products.  P, in units where the running
// maximum is 2^7 (at most 2^15 until it is moved), is rounded to f16: 2^−11 relative, and
// what lies below f16's range is less than 2^−32 of the largest.
//
// Work units are blocks of 128 keys of one (sequence, key head, row tile), dealt out evenly
// as in cache_attn.cu, and the parts of a tile are joined by the same second kernel.  In a
// CTA one warp loads, the others take 16 keys of every block each, with a maximum, sum and O
// of their own that meet in shared memory at the end of a tile.
#include "cache_join.cuh"
#include "fp8_device.cuh"

namespace attn {
namespace {

constexpr float kShift = 7.0f;  // log2 of P where a score is the reference maximum
constexpr float kTau = 8.0f;    // log2: the reference moves when exceeded by more

struct CacheAttnFp8Params {
  CacheAttnParams a;
  Fp8Pages f;
  const uint16_t* q;
  const uint16_t* kn;
  const uint16_t* vn;
  long long q_st[2], kn_st[2], vn_st[2];
};

// The blocks of 128 cached keys; the new tokens go with the last.
struct RowsPlan {
  static __device__ __forceinline__ KeyPlan of(const CacheAttnParams& p, int s) {
    KeyPlan k;
    const SeqRows r = seq_rows(p.c, s);
    k.q0 = r.q0;
    k.n = min(r.n, p.c.max_new);
    k.len = seq_len(p.c, s);
    k.nfull = k.len >> 7;
    k.tail = k.len & 127;
    k.off = 0;
    k.db = max((k.len + 127) >> 7, 1) - 1;
    return k;
  }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int D, int NT>
struct FL {
  static constexpr int kWarps = 8;                       // of 16 keys each
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr uint32_t kKeys = 128u * D;            // bytes of a block's K or V
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kRing = 0;                   // [stage][K, V]
  static constexpr int kPitch = D + 8;                   // floats a row of a warp's O: no bank conflicts
  static constexpr uint32_t kMerge = kStages * 2 * kKeys;        // [warp][8 rows][kPitch]
  static constexpr uint32_t kMl = kMerge + kWarps * 8 * kPitch * 4;  // [warp][8 NT] reference maximum and sum
  static constexpr uint32_t kScales = kMl + kWarps * 8 * NT * 8;     // [stage][8 of K, 8 of V]
  static constexpr uint32_t kBar = kScales + kStages * 16;
  static constexpr uint32_t kMisc = kBar + 8 * 2 * kStages;  // abort flag
  static constexpr uint32_t kSums = kMisc + 8;
  static constexpr uint32_t kTable = (kSums + 4 * (kWarps + 1) + 15) & ~15u;
  static constexpr uint32_t kBytes = kTable + 1024;      // + alignment; the table comes on top
};

// Where 16-byte chunk c of row r lies in a tile of rows of D bytes, as TMA's swizzle of
// 128 (64) bytes puts it.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}
// Key of fragment row g: two rows that are read together have to differ in the bit that
// picks the half of the 32 banks.
template <int D>
__device__ __forceinline__ int key_of(int g) {
  return D == 128 ? (g >> 1) | ((g & 1) << 2) : g;
}

template <int D, int NT>
__global__ void __launch_bounds__(FL<D, NT>::kThreads, 1)
    cache_attn_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const CacheAttnFp8Params fp) {
  using L = FL<D, NT>;
  const CacheAttnParams& p = fp.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  auto full = [&](int s) { return base + L::kBar + 8u * s; };
  auto empty = [&](int s) { return base + L::kBar + 8u * (L::kStages + s); };
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  int* const tab = reinterpret_cast<int*>(smem + L::kTable);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), L::kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  prefix_table(p.c.n_seq, tab, reinterpret_cast<int*>(smem + L::kSums),
               [&](int s) { return units_of<RowsPlan>(p, s); });
  const int units = tab[p.c.n_seq];
  if (cta == 0)
    for (int i = threadIdx.x; i <= p.c.n_seq; i += L::kThreads) p.ws_table[i] = tab[i];
  const int grid = min(static_cast<int>(gridDim.x), units);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (cta >= grid) return;
  const int u0 = range_start(units, cta, grid), u1 = range_start(units, cta + 1, grid);
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (warp == L::kWarps) {
    // ============================================================= loader
    // Lane i < 8 copies the keys of the block's i-th 16 slots (with those behind them, as
    // many as a copy holds) and lane 8 + i their values; both fetch the scale as well.
    int g = 0, copies = 0;
    bool ok = true;
    const int i16 = lane & 7, ps = p.piece;
    const bool is_v = lane >= 8;
    for (int u = u0; u < u1 && ok;) {
      const Segment sg = segment_at<RowsPlan>(p, tab, u, u1);
      u += sg.b1 - sg.b0;
      int page_next = 0, slot_next = 0;  // of the block after the next
      auto locate = [&](int b) {
        const int j = (b << 7) + 16 * i16;
        const int blk = j / p.c.page_size;
        slot_next = j - blk * p.c.page_size;
        page_next = lane < 16 && j < sg.k.len ? page_for_read(p.c, sg.s, blk) : 0;
      };
      auto scale_of = [&](int b, int page, int slot) -> uint8_t {
        if (lane >= 16 || (b << 7) + 16 * i16 >= sg.k.len) return 0;
        return (is_v ? fp.f.vs : fp.f.ks)[(static_cast<long long>(page) * p.c.hkv + sg.h) * fp.f.per + (slot >> 4)];
      };
      locate(sg.b0);
      int page = page_next, slot = slot_next;
      uint8_t scale = scale_of(sg.b0, page, slot);
      if (sg.b0 + 1 < sg.b1) locate(sg.b0 + 1);
      for (int b = sg.b0; b < sg.b1 && ok; ++b, ++g) {
        const int st = g % L::kStages, ph = (g / L::kStages) & 1;
        const int cv = min(sg.k.len - (b << 7), 128), npc = (cv + ps - 1) / ps;
        int got = 1;
        if (lane == 0) got = wait_bar(empty(st), ph ^ 1u, wc) && !(p.test_flags & 1u);
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        __syncwarp();
        if (lane < 16) smem[L::kScales + st * 16 + lane] = scale;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full(st), static_cast<uint32_t>(max(npc, 0) * ps) * 2u * D);
        __syncwarp();
        if (lane < 16 && 16 * i16 < cv && (16 * i16) % ps == 0)
          tma_load_4d(base + L::kRing + (2 * st + (is_v ? 1 : 0)) * L::kKeys + 16 * i16 * D, is_v ? &tm_v : &tm_k, 0, sg.h,
                      slot, page, full(st));
        __syncwarp();
        ++copies;
        page = page_next;
        slot = slot_next;
        if (b + 1 < sg.b1) scale = scale_of(b + 1, page, slot);
        if (b + 2 < sg.b1) locate(b + 2);
      }
    }
    // No copy may be in flight when the CTA ends, whatever ended the loop.
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      for (int n = max(0, copies - L::kStages); n < copies; ++n)
        while (!mbar_try_wait(full(n % L::kStages), (n / L::kStages) & 1u))
          if (globaltimer_ns() - t0 > p.timeout_ns) break;
    }
    return;
  }

  // ================================================================== the sums
  const int gr = lane >> 2, t4 = lane & 3;
  const int grp = p.c.group, H = p.c.hkv * grp;
  constexpr int kSteps = D / 16;  // m16n8k16 products of a score tile, and tiles of Oᵀ
  // Places in a warp's 16 rows of K and V.
  uint32_t k_at[2][D / 64], v_at[D / 32];
#pragma unroll
  for (int hf = 0; hf < D / 64; ++hf) {
    k_at[0][hf] = chunk_at<D>(16 * warp + key_of<D>(gr), 4 * hf + t4);
    k_at[1][hf] = chunk_at<D>(16 * warp + 8 + key_of<D>(gr), 4 * hf + t4);
  }
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    v_at[c] = L::kKeys + chunk_at<D>(16 * warp + (lane & 8) + key_of<D>(lane & 7), 2 * c + (lane >> 4));

  int g = 0;
  bool ok = true;
  for (int u = u0; u < u1;) {
    const Segment sg = segment_at<RowsPlan>(p, tab, u, u1);
    const bool first_of_cta = u == u0;
    u += sg.b1 - sg.b0;
    const int row0 = sg.m * p.rows, n_rows = min(sg.k.n * grp - row0, p.rows);
    // ---- Q: the rows of this thread's fragments (row gr of each tile), as f16
    uint32_t qf[NT][kSteps][2];
    float mult[NT][2];  // of the scores in its columns (rows 2·t4 and 2·t4 + 1)
    auto q_row = [&](int r) {
      const int rr = row0 + min(r, n_rows - 1);
      return fp.q + (sg.k.q0 + rr / grp) * fp.q_st[0] + (sg.h * grp + rr % grp) * fp.q_st[1];
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
        for (int i = 0; i < 8; ++i)
          qf[nt][4 * hf + i / 2][i & 1] =
              pack_f16x2(__uint_as_float(w[hf][i] << 16) * f, __uint_as_float(w[hf][i] & 0xFFFF0000u) * f);
      const float rest = up == 127 ? 0.5f * inv : inv;  // (2^−127 is no normal number)
      mult[nt][0] = __shfl_sync(0xffffffffu, rest, 8 * t4);
      mult[nt][1] = __shfl_sync(0xffffffffu, rest, 8 * t4 + 4);
    }
    float o[NT][kSteps][4], m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][c][i] = 0.f;
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = 0.f;
    }
    // Scores (log2 units; −inf where a row does not see a key) to P: a reference that is
    // exceeded by more than kTau moves, and with it O and the sums.
    auto weigh = [&](float(&s)[NT][4]) {
      bool need = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[nt][i] = fmaxf(s[nt][i], s[nt][i + 2]);
          need = need || mx[nt][i] > m_run[nt][i] + kTau || (m_run[nt][i] == -INFINITY && mx[nt][i] > -INFINITY);
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = mx[nt][i];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            if (m > m_run[nt][i]) {
              const float alpha = ex2_mufu(m_run[nt][i] - m);
              m_run[nt][i] = m;
              l_run[nt][i] *= alpha;
#pragma unroll
              for (int c = 0; c < kSteps; ++c) {
                o[nt][c][i] *= alpha;
                o[nt][c][i + 2] *= alpha;
              }
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = m_run[nt][i & 1];
          s[nt][i] = ex2_mufu(s[nt][i] - (m == -INFINITY ? 0.f : m - kShift));
          l_run[nt][i & 1] += s[nt][i];
        }
    };

    for (int b = sg.b0; b < sg.b1; ++b, ++g) {
      const int st = g % L::kStages;
      ok = ok && wait_bar(full(st), (g / L::kStages) & 1, wc);
      ok = !__any_sync(0xffffffffu, !ok);
      const int nv = min(sg.k.len - (b << 7) - 16 * warp, 16);  // keys of this warp
      if (ok && nv > 0) {
        const uint32_t tile = base + L::kRing + 2 * st * L::kKeys;
        const float ka = power_of(scale_byte(smem[L::kScales + st * 16 + warp]));
        const float vb = power_of(scale_byte(smem[L::kScales + st * 16 + 8 + warp]));
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          uint32_t lo[4], hi[4];
          ld_shared_v4(tile + k_at[0][hf], lo);
          ld_shared_v4(tile + k_at[1][hf], hi);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(lo[j]), e4m3x2_to_f16x2(hi[j]), e4m3x2_to_f16x2(lo[j] >> 16),
                                   e4m3x2_to_f16x2(hi[j] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a, qf[nt][4 * hf + j][0], qf[nt][4 * hf + j][1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[nt][i] = s[nt][i] * mult[nt][i & 1] * ka;
            if (nv < 16 && key_of<D>(gr) + (i & 2 ? 8 : 0) >= nv) s[nt][i] = -INFINITY;
          }
        weigh(s);
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pf[nt][0] = transposed(pack_f16x2(s[nt][0], s[nt][1]));
          pf[nt][1] = transposed(pack_f16x2(s[nt][2], s[nt][3]));
        }
        // Codes behind the sequence's end: their P is 0, but a NaN would spread.
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (nv < 16) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            keep[x] = (key_of<D>(2 * t4) + 8 * x < nv ? 0xffffu : 0u) |
                      (key_of<D>(2 * t4 + 1) + 8 * x < nv ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[4];
          ldmatrix_x4_trans(tile + v_at[c], r);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            // (key 2t, value 2g), (2t, 2g + 1), (2t + 1, 2g), (2t + 1, 2g + 1) → pairs of keys
            const uint32_t w0 = __byte_perm(r[2 * y] & keep[0], 0u, 0x3120), w1 = __byte_perm(r[2 * y + 1] & keep[1], 0u, 0x3120);
            const uint32_t a[4] = {e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w0 >> 16), e4m3x2_to_f16x2(w1),
                                   e4m3x2_to_f16x2(w1 >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float pv[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(pv, a, pf[nt][0], pf[nt][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[nt][2 * c + y][i] = fmaf(pv[i], vb, o[nt][2 * c + y][i]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(empty(st));
    }
    // ---- the new tokens' own keys, 16 a warp from the last on (whose cached keys are often none)
    const int k0 = 16 * (L::kWarps - 1 - warp);
    if (ok && sg.b1 == sg.k.db + 1 && k0 < sg.k.n) {
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
      const uint16_t* const kn = fp.kn + static_cast<long long>(sg.h) * fp.kn_st[1];
      const uint16_t* const vn = fp.vn + static_cast<long long>(sg.h) * fp.vn_st[1];
      const int ja = k0 + gr, jb = ja + 8;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
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
          mma_bf16(s[nt], a0, q.x, q.y);
          mma_bf16(s[nt], a1, q.z, q.w);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t see[2] = {__shfl_sync(0xffffffffu, mine, 8 * nt + 2 * t4),
                                 __shfl_sync(0xffffffffu, mine, 8 * nt + 2 * t4 + 1)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[nt][i] = (see[i & 1] >> (gr + (i & 2 ? 8 : 0))) & 1u ? s[nt][i] * p.scale_log2 : -INFINITY;
      }
      weigh(s);
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pf[nt][0] = transposed(pack_bf16x2(s[nt][0], s[nt][1]));
        pf[nt][1] = transposed(pack_bf16x2(s[nt][2], s[nt][3]));
      }
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = k0 + 2 * t4 + (x & 1) + (x & 2 ? 8 : 0);
          w[x] = j < sg.k.n
                     ? *reinterpret_cast<const uint32_t*>(vn + (sg.k.q0 + j) * fp.vn_st[0] + 16 * c + 2 * gr)
                     : 0u;
        }
        const uint32_t a[4] = {__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                               __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][c], a, pf[nt][0], pf[nt][1]);
      }
    }
    // ---- the warps' sums meet
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = l_run[nt][i];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        if (gr == 0)
          reinterpret_cast<float2*>(smem + L::kMl)[warp * 8 * NT + 8 * nt + 2 * t4 + i] =
              make_float2(m_run[nt][i] == -INFINITY ? -INFINITY : m_run[nt][i] - kShift, l);
      }
    const bool whole = sg.b0 == 0 && sg.b1 == sg.k.db + 1;
    const int slot = 2 * cta + (first_of_cta ? 0 : 1);
    float* const merge = reinterpret_cast<float*>(smem + L::kMerge);
    constexpr int kPer = D / 32;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (8 * nt >= n_rows) break;  // (the same for all warps)
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(merge + (warp * 8 + 2 * t4 + i) * L::kPitch + 16 * c + 2 * gr) =
              make_float2(o[nt][c][i], o[nt][c][i + 2]);
      asm volatile("bar.sync 1, %0;" ::"n"(32 * L::kWarps) : "memory");
      // Warp w joins row w: its lanes kPer values each.
      const int r = 8 * nt + warp;
      if (r < n_rows && ok) {
        const float2* const ml = reinterpret_cast<const float2*>(smem + L::kMl) + r;
        float mx = -INFINITY, sum = 0.f, acc[kPer] = {};
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) mx = fmaxf(mx, ml[w * 8 * NT].x);
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) {
          const float2 x = ml[w * 8 * NT];
          const float f = x.x == -INFINITY ? (x.y != x.y ? x.y : 0.f) : ex2_mufu(x.x - mx);
          sum += f * x.y;
          const float* const src = merge + (w * 8 + warp) * L::kPitch + lane * kPer;
#pragma unroll
          for (int i = 0; i < kPer; ++i) acc[i] += f * src[i];
        }
        if (whole) {
          const int rr = row0 + r, hq = sg.h * grp + rr % grp;
          const long long token = sg.k.q0 + rr / grp;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          uint16_t* const dst = p.o + (token * H + hq) * D + lane * kPer;
          if constexpr (kPer == 4)
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
          else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
          if (lane == 0)
            p.lse[static_cast<long long>(hq) * p.c.total + token] =
                sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.69314718055994531f;
        } else {
          const long long part = static_cast<long long>(slot) * p.rows + r;
          float* const dst = p.ws_o + part * D + lane * kPer;
          if constexpr (kPer == 4) *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          else *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
          if (lane == 0) p.ws_ml[part] = make_float2(mx, sum);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * L::kWarps) : "memory");
    }
  }
}

template <int D, int NT>
cudaError_t launch(const CacheAttnFp8Launch& a) {
  using L = FL<D, NT>;
  CacheAttnFp8Params p = {a.p, a.f, a.q, a.kn, a.vn, {a.q_st[0], a.q_st[1]}, {a.kn_st[0], a.kn_st[1]}, {a.vn_st[0], a.vn_st[1]}};
  const unsigned int smem = L::kBytes + 4u * (p.a.c.n_seq + 1);
  static volatile bool configured[64] = {};
  if (a.device < 0 || a.device >= 64) return cudaErrorInvalidDevice;
  if (!configured[a.device]) {
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_fp8_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               L::kBytes + 4 * (kCacheMaxSeq + 1));
    if (e != cudaSuccess) return e;
    configured[a.device] = true;
  }
  cache_attn_fp8_kernel<D, NT><<<a.grid, L::kThreads, smem, a.stream>>>(a.k, a.v, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<D, RowsPlan>(p.a, a.grid, a.stream);
}

}  // namespace

cudaError_t launch_cache_attn_fp8(const CacheAttnFp8Launch& a) {
  if (a.p.c.d == 64) return a.p.rows > 8 ? launch<64, 2>(a) : launch<64, 1>(a);
  return a.p.rows > 8 ? launch<128, 2>(a) : launch<128, 1>(a);
}

}  // namespace attn
