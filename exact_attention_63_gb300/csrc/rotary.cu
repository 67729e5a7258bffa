// Rotary positions on q and k, forward and inverse.
//
// A turn of a pair (u, w) by a = position·inv_freq.  What matters of a is its fraction of a
// turn: inv_freq/2π as a 64-bit fraction of a turn, times the position in integers, is that
// fraction modulo 1 with an error of position·2^−64 (and fp64's own 2^−53 of the frequency),
// where a product in fp32 would be off by 0.06 radians at position 10^6.
//   Bound by memory: every element is read and written once.  The sines of a row serve all
// of its heads: a CTA puts those of its rows into shared memory, then its threads take
// 2·VEC elements at a time, whichever row, tensor and head they belong to.
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "attn_device.cuh"
#include "attn_gb300.h"
#include "attn_launch.h"
#include "cache_launch.h"

namespace {

constexpr int kThreads = 256;

struct RotaryParams {
  const uint16_t* x[2];
  uint16_t* y[2];
  long long x_st[2][3], y_st[2][3];  // batch, row, head
  int heads[2];
  const int* positions;              // may be null
  long long pos_st;
  const double* inv_freq;
  int batch, rows, part, per_cta;    // rows of a CTA
  float magnitude;
  int inverse;
  attn::FastDiv by_rows, by_heads;   // by_heads: both tensors' heads
};

template <int BYTES> struct Vec;
template <> struct Vec<2> { using T = uint16_t; };
template <> struct Vec<4> { using T = uint32_t; };
template <> struct Vec<8> { using T = uint2; };
template <> struct Vec<16> { using T = uint4; };

template <int VEC>
struct Bits {
  uint16_t v[VEC];
};
template <int VEC>
__device__ __forceinline__ Bits<VEC> load(const uint16_t* p) {
  using T = typename Vec<2 * VEC>::T;
  union { T t; Bits<VEC> b; } u;
  u.t = *reinterpret_cast<const T*>(p);
  return u.b;
}
template <int VEC>
__device__ __forceinline__ void store(uint16_t* p, const Bits<VEC>& x) {
  using T = typename Vec<2 * VEC>::T;
  union { T t; Bits<VEC> b; } u;
  u.b = x;
  *reinterpret_cast<T*>(p) = u.t;
}
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// VEC: elements of an access, the largest power of two up to 8 that divides part/2.
template <int D, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 5) rotary_kernel(const RotaryParams p) {
  // [per_cta][VEC][part / 2 / VEC]: lanes read neighbouring runs of VEC pairs, the same pair of each at
  // a time (in the pairs' own order they met in banks, four at a time).
  extern __shared__ float2 turns[];
  const int first = blockIdx.x * p.per_cta, n = min(p.per_cta, p.batch * p.rows - first), half = p.part / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int r = i / half, f = i - r * half, row = first + r, b = p.by_rows(row), at = row - b * p.rows;
    const int pos = p.positions != nullptr ? p.positions[b * p.pos_st + at] : at;
    // A position's fraction of a turn, then the position's own, modulo 1 in units of 2^−64.
    const double t = p.inv_freq[f] * 0.15915494309189533577;
    const unsigned long long unit = static_cast<unsigned long long>(__double2ll_rn((t - rint(t)) * 9223372036854775808.0)) << 1;
    const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * unit;
    const float half_turns = static_cast<float>(static_cast<long long>(turn)) * 1.0842021724855044e-19f;  // 2^−63
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    turns[r * half + f % VEC * (half / VEC) + f / VEC] = make_float2(cs * p.magnitude, (p.inverse ? -sn : sn) * p.magnitude);
  }
  __syncthreads();
  constexpr int kItems = D / (2 * VEC);  // of a head
  const int heads = p.heads[0] + p.heads[1], items = n * heads * kItems, turned = half / VEC;
#pragma unroll 2
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int c = i % kItems, rh = i / kItems, r = p.by_heads(rh), hh = rh - r * heads;
    const int row = first + r, b = p.by_rows(row), at = row - b * p.rows;
    const int which = hh >= p.heads[0], h = which ? hh - p.heads[0] : hh;
    const uint16_t* const x = p.x[which] + b * p.x_st[which][0] + at * p.x_st[which][1] + h * p.x_st[which][2];
    uint16_t* const y = p.y[which] + b * p.y_st[which][0] + at * p.y_st[which][1] + h * p.y_st[which][2];
    const bool turn = c < turned;
    const int lo = INTERLEAVED || !turn ? 2 * VEC * c : VEC * c, hi = INTERLEAVED || !turn ? lo + VEC : lo + half;
    if (!turn && x == y) continue;
    Bits<VEC> u = load<VEC>(x + lo), w = load<VEC>(x + hi);
    if (turn) {
      const float2* const cs = turns + r * half + c;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 t = cs[e * (half / VEC)];
        // pair e: (u[e], w[e]), or neighbours in (u, w)
        uint16_t& a = !INTERLEAVED ? u.v[e] : (2 * e < VEC ? u.v[2 * e] : w.v[2 * e - VEC]);
        uint16_t& z = !INTERLEAVED ? w.v[e] : (2 * e + 1 < VEC ? u.v[2 * e + 1] : w.v[2 * e + 1 - VEC]);
        const float fa = to_f32(a), fz = to_f32(z);
        const uint32_t both = attn::pack_bf16x2(fa * t.x - fz * t.y, fz * t.x + fa * t.y);
        a = static_cast<uint16_t>(both);
        z = static_cast<uint16_t>(both >> 16);
      }
    }
    store<VEC>(y + lo, u);
    store<VEC>(y + hi, w);
  }
}

template <int D, int VEC>
void launch(const RotaryParams& p, bool interleaved, unsigned int blocks, unsigned int smem, cudaStream_t stream) {
  if (interleaved) rotary_kernel<D, VEC, true><<<blocks, kThreads, smem, stream>>>(p);
  else rotary_kernel<D, VEC, false><<<blocks, kThreads, smem, stream>>>(p);
}
template <int D>
void launch(const RotaryParams& p, bool interleaved, unsigned int blocks, unsigned int smem, cudaStream_t stream) {
  const int half = p.part / 2;
  if (half % 8 == 0) launch<D, 8>(p, interleaved, blocks, smem, stream);
  else if (half % 4 == 0) launch<D, 4>(p, interleaved, blocks, smem, stream);
  else if (half % 2 == 0) launch<D, 2>(p, interleaved, blocks, smem, stream);
  else launch<D, 1>(p, interleaved, blocks, smem, stream);
}

int describe(const attn_rows* t, int rows, int d, int which, RotaryParams* p) {
  if (t->struct_size < sizeof(attn_rows)) return ATTN_ERR_LAYOUT;
  if (t->x == nullptr || t->y == nullptr) return ATTN_ERR_NULL;
  if (t->heads < 1 || t->heads > 65536) return ATTN_ERR_SHAPE;
  const long long hd = static_cast<long long>(t->heads) * d, dense[3] = {hd * rows, hd, d};
  for (int side = 0; side < 2; ++side) {
    const long long* const in = side ? t->y_strides : t->x_strides;
    const bool zero = in[0] == 0 && in[1] == 0 && in[2] == 0;
    for (int i = 0; i < 3; ++i) {
      if (!zero && (in[i] <= 0 || (in[i] & 7) != 0 || in[i] >= (1ll << 38))) return ATTN_ERR_LAYOUT;
      (side ? p->y_st : p->x_st)[which][i] = zero ? dense[i] : in[i];
    }
  }
  if (((reinterpret_cast<uintptr_t>(t->x) | reinterpret_cast<uintptr_t>(t->y)) & 15) != 0) return ATTN_ERR_ALIGN;
  p->x[which] = static_cast<const uint16_t*>(t->x);
  p->y[which] = static_cast<uint16_t*>(t->y);
  p->heads[which] = t->heads;
  return ATTN_OK;
}

}  // namespace

extern "C" int attn_rotary(const attn_rows* q, const attn_rows* k, int batch, int rows, int d, const int* positions,
                           long long positions_stride, const double* inv_freq, int rotary_dim, int interleaved,
                           float magnitude, int inverse, cudaStream_t stream) {
  if (q == nullptr || inv_freq == nullptr) return ATTN_ERR_NULL;
  if (batch < 1 || rows < 1 || static_cast<long long>(batch) * rows > (1ll << 30)) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (rotary_dim < 2 || rotary_dim > d || (rotary_dim & 1) != 0 || positions_stride < 0) return ATTN_ERR_LAYOUT;
  if (!std::isfinite(magnitude)) return ATTN_ERR_SCALE;
  RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  int rc = describe(q, rows, d, 0, &p);
  if (rc != ATTN_OK || (k != nullptr && (rc = describe(k, rows, d, 1, &p)) != ATTN_OK)) return rc;
  if ((reinterpret_cast<uintptr_t>(positions) & 3) != 0 || (reinterpret_cast<uintptr_t>(inv_freq) & 7) != 0)
    return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  if ((rc = attn::usable_device(&dev, &status, &sms)) != ATTN_OK) return rc;
  p.positions = positions;
  p.pos_st = positions_stride;
  p.inv_freq = inv_freq;
  p.batch = batch;
  p.rows = rows;
  p.part = rotary_dim;
  p.magnitude = magnitude;
  p.inverse = inverse != 0;
  p.by_rows = attn::fast_div(rows);
  p.by_heads = attn::fast_div(p.heads[0] + p.heads[1]);
  const long long all = static_cast<long long>(batch) * rows;
  p.per_cta = all >= 16ll * sms ? 4 : 1;
  const unsigned int blocks = static_cast<unsigned int>((all + p.per_cta - 1) / p.per_cta);
  const unsigned int smem = static_cast<unsigned int>(p.per_cta * rotary_dim / 2 * sizeof(float2));
  if (d == 64) launch<64>(p, interleaved != 0, blocks, smem, stream);
  else launch<128>(p, interleaved != 0, blocks, smem, stream);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e, "rotary launch");
}
