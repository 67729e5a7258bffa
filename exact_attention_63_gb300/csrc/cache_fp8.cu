// Rows into and out of a cache of E4M3 codes.  Both are bound by memory: 2 bytes an element
// on the bf16 side, 1 on the cache's.
#include "attn_gb300.h"
#include "cache_device.cuh"
#include "fp8_device.cuh"

namespace attn {
namespace {

// The last entry s of an ascending list of n with at(s) <= x, by a whole warp: 32
// candidates a step.
template <class F>
__device__ __forceinline__ int find_warp(int n, long long x, int lane, F at) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool le = lane * step < n && at(lo + lane * step) <= x;
    const unsigned int votes = __ballot_sync(0xffffffffu, le);
    const int k = votes == 0u ? 0 : 31 - __clz(votes);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// ------------------------------------------------------------------- append
// Work is dealt out by block of 16 slots: a warp takes one key head's k or v in one block,
// so the block's scale and the rows that need it are one warp's.  Sequence s owns the
// blocks' numbers from cu[s]/16 + 2s on: n rows touch at most n/16 + 2 blocks, so the
// numbers of two sequences never meet and the host needs no lengths.
//   A lane holds 8 elements of 2 (d = 128) or 4 rows at a time; all 16 rows are in flight.
template <int D>
__global__ void __launch_bounds__(256, 4) cache_append_fp8_kernel(const CacheAppendFp8Params p, int items) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kSteps = 16 / kAtOnce;  // lanes a row, rows a step
  const CacheParams& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long wi = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const long long unit = wi / items;
  const int item = static_cast<int>(wi - unit * items), h = item >> 1, which = item & 1;
  auto base = [&](int s) { return (static_cast<long long>(min(max(c.cu[s], 0), p.n_rows)) >> 4) + 2ll * s; };
  const int s = find_warp(c.n_seq, unit, lane, base);
  const int a = min(max(c.cu[s], 0), p.n_rows), z = min(max(c.cu[s + 1], a), p.n_rows);
  const int len = seq_len(c, s), first = len - (z - a);  // (may be negative: those slots are skipped)
  const long long nth = unit - base(s);
  if (nth < 0) return;
  const long long blk = (max(first, 0) >> 4) + nth;
  if (blk * 16 >= len || z == a) return;
  const int slot0 = static_cast<int>(blk) * 16, page_no = slot0 / c.page_size, in = slot0 - page_no * c.page_size;
  const int page = c.table[static_cast<long long>(s) * c.max_blocks + page_no];
  if (page < 0 || page >= c.n_pages) return;

  const long long* const st = which ? c.v_st : c.k_st;
  const long long* const ns = which ? p.vn_st : p.kn_st;
  uint8_t* const dst = (which ? p.f.v : p.f.k) + page * st[0] + in * st[1] + h * st[2] + (lane % kLanes) * 8;
  const uint16_t* const from = (which ? p.vn : p.kn) + h * ns[1] + (lane % kLanes) * 8;
  uint8_t* const scale = (which ? p.f.vs : p.f.ks) + (static_cast<long long>(page) * c.hkv + h) * p.f.per + (in >> 4);

  uint4 x[kSteps];
  uint32_t there = 0u;  // rows of this lane's that are new
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = slot0 + i * kAtOnce + lane / kLanes;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= first && slot < len) {
      const int at = a + (slot - first), src = p.rows != nullptr ? p.rows[at] : at;
      if (src >= 0 && src < c.total) {
        x[i] = *reinterpret_cast<const uint4*>(from + src * ns[0]);
        there |= 1u << i;
      }
    }
  }
  const bool kept = slot0 < first;  // older rows stay in this block
  const int old = kept ? scale_byte(*scale) : kFp8Lowest;
  // The largest |x|: bf16 bits without the sign are ordered like their values; infinities
  // and NaN, above all numbers, are looked for only if the largest is one of them.
  auto largest = [&](bool finite) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u = w[e] & 0x7FFF7FFFu, lo = u & 0xFFFFu, hi = u >> 16;
        m = max(m, finite && lo >= 0x7F80u ? 0u : lo);
        m = max(m, finite && hi >= 0x7F80u ? 0u : hi);
      }
    }
    return __reduce_max_sync(0xffffffffu, m);
  };
  if (!__any_sync(0xffffffffu, there != 0u)) return;
  uint32_t top = largest(false);
  if (top >= 0x7F80u) top = largest(true);
  const int e = max(byte_for(top), old);
  if (kept && e > old) {  // older rows in units of the new scale
    const float f = power_of(max(127 + old - e, 1));  // (2^−126 and less leave nothing of a code)
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = i * kAtOnce + lane / kLanes;
      if (slot0 + r >= first) continue;
      uint2* const at = reinterpret_cast<uint2*>(dst + r * st[1]);
      const uint2 w = *at;
      uint32_t out[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = k ? w.y : w.x;
        float v0, v1, v2, v3;
        f16x2_to_f32(e4m3x2_to_f16x2(u & 0xFFFFu), v0, v1);
        f16x2_to_f32(e4m3x2_to_f16x2(u >> 16), v2, v3);
        out[k] = to_e4m3x2(v0 * f, v1 * f) | (to_e4m3x2(v2 * f, v3 * f) << 16);
      }
      *at = make_uint2(out[0], out[1]);
    }
  }
  const float inv = power_of(254 - e);  // 2^−(e − 127): x times it is exact or far below the codes' smallest
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (!((there >> i) & 1u)) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t two[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      two[k] = to_e4m3x2(__uint_as_float(w[k] << 16) * inv, __uint_as_float(w[k] & 0xFFFF0000u) * inv);
    *reinterpret_cast<uint2*>(dst + (i * kAtOnce + lane / kLanes) * st[1]) =
        make_uint2(two[0] | (two[1] << 16), two[2] | (two[3] << 16));
  }
  if (lane == 0 && (!kept || e > old)) *scale = static_cast<uint8_t>(e);
}

// ------------------------------------------------------------------- gather
// A warp writes one token's k or v, 8 elements a lane, four pieces in flight.
template <int D>
__global__ void __launch_bounds__(256) cache_gather_fp8_kernel(const CacheGatherFp8Params p) {
  constexpr int kLanes = D / 8;
  const CacheParams& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long wi = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int i = static_cast<int>(wi >> 1), which = static_cast<int>(wi & 1);
  if (i >= c.total) return;
  const int s = find_warp(c.n_seq, i, lane, [&](int x) { return static_cast<long long>(c.cu[x]); });
  const SeqRows r = seq_rows(c, s);
  if (i < r.q0 || i >= r.q0 + r.n) return;
  const int slot = seq_len(c, s) - r.n + (i - r.q0);
  if (slot < 0) return;
  const int blk = slot / c.page_size, in = slot - blk * c.page_size;
  const int page = page_for_read(c, s, blk);
  const long long* const st = which ? c.v_st : c.k_st;
  const uint8_t* const from = (which ? p.f.v : p.f.k) + page * st[0] + in * st[1];
  const uint8_t* const scale = (which ? p.f.vs : p.f.ks) + static_cast<long long>(page) * c.hkv * p.f.per + (in >> 4);
  uint16_t* const to = (which ? p.v_out : p.k_out) + static_cast<long long>(i) * c.hkv * D;
  const int pieces = c.hkv * kLanes;
  for (int q = lane; q < pieces; q += 128) {
    uint2 x[4];
    uint8_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = q + 32 * e, h = at / kLanes;
      if (at < pieces) {
        x[e] = *reinterpret_cast<const uint2*>(from + h * st[2] + (at % kLanes) * 8);
        b[e] = scale[static_cast<long long>(h) * p.f.per];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = q + 32 * e;
      if (at >= pieces) continue;
      const float f = power_of(scale_byte(b[e]));
      uint32_t out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        f16x2_to_f32(e4m3x2_to_f16x2((k & 2 ? x[e].y : x[e].x) >> (k & 1 ? 16 : 0)), lo, hi);
        out[k] = pack_bf16x2(lo * f, hi * f);
      }
      *reinterpret_cast<uint4*>(to + at * 8) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

}  // namespace

cudaError_t launch_cache_append_fp8(const CacheAppendFp8Params& p, cudaStream_t stream) {
  const long long units = p.n_rows / 16 + 2ll * p.c.n_seq, items = 2ll * p.c.hkv;
  const unsigned int blocks = static_cast<unsigned int>((units * items + 7) / 8);
  if (p.c.d == 64) cache_append_fp8_kernel<64><<<blocks, 256, 0, stream>>>(p, static_cast<int>(items));
  else cache_append_fp8_kernel<128><<<blocks, 256, 0, stream>>>(p, static_cast<int>(items));
  return cudaGetLastError();
}

cudaError_t launch_cache_gather_fp8(const CacheGatherFp8Params& p, cudaStream_t stream) {
  const unsigned int blocks = static_cast<unsigned int>((2ll * p.c.total + 7) / 8);
  if (p.c.d == 64) cache_gather_fp8_kernel<64><<<blocks, 256, 0, stream>>>(p);
  else cache_gather_fp8_kernel<128><<<blocks, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
