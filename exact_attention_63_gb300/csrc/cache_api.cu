// C ABI of the cache operators: argument checks, TMA descriptors, launches.
// Declarations and their contracts are in include/attn_gb300.h.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_gb300.h"
#include "attn_launch.h"
#include "cache_launch.h"

namespace {

using attn::CacheParams;

constexpr unsigned int kDefaultTimeoutMs = 4000;
constexpr long long kMaxCapacity = 1ll << 30;
constexpr long long kMaxInt = 0x7FFFFFFFll;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// All zero → dense; else positive multiples of 8 (`unit`: of 16 for elements of a byte)
// below 2^38 (TMA: 16-byte multiples below 2^40 bytes).
template <int N>
bool resolve(const long long in[N], const long long dense[N], long long out[N], int unit = 8) {
  bool zero = true;
  for (int i = 0; i < N; ++i) zero = zero && in[i] == 0;
  for (int i = 0; i < N; ++i) {
    if (!zero && (in[i] <= 0 || (in[i] & (unit - 1)) != 0 || in[i] >= (1ll << 38))) return false;
    out[i] = zero ? dense[i] : in[i];
  }
  return true;
}

// The cache's fields that every operator needs; k and v where `kv` says so
// (bit 0: k, bit 1: v), in strides of multiples of `unit` elements.
int check_cache(const attn_cache* a, int kv, CacheParams* c, int unit = 8) {
  if (a == nullptr) return ATTN_ERR_NULL;
  if (a->struct_size < sizeof(attn_cache)) return ATTN_ERR_CACHE;
  if (a->block_table == nullptr || ((kv & 1) && a->k == nullptr) || ((kv & 2) && a->v == nullptr)) return ATTN_ERR_NULL;
  if (a->n_pages < 1 || a->max_blocks < 1 || a->n_seq < 1 || a->num_kv_heads < 1) return ATTN_ERR_SHAPE;
  if (kv != 0 && a->d != 64 && a->d != 128) return ATTN_ERR_HEAD_DIM;
  if (a->page_size < 16 || a->page_size > 65536 || a->page_size % 16 != 0 || a->n_seq > attn::kCacheMaxSeq ||
      static_cast<long long>(a->max_blocks) * a->page_size > kMaxCapacity)
    return ATTN_ERR_CACHE;
  std::memset(c, 0, sizeof(*c));
  const long long hd = static_cast<long long>(a->num_kv_heads) * a->d;
  const long long dense[3] = {hd * a->page_size, hd, a->d};
  if ((kv & 1) && !resolve<3>(a->k_strides, dense, c->k_st, unit)) return ATTN_ERR_CACHE;
  if ((kv & 2) && !resolve<3>(a->v_strides, dense, c->v_st, unit)) return ATTN_ERR_CACHE;
  if (((kv & 1) && !aligned(a->k, 16)) || ((kv & 2) && !aligned(a->v, 16)) || !aligned(a->weights, 16) ||
      !aligned(a->positions, 16) || !aligned(a->block_table, 4) || !aligned(a->seq_lens, 4))
    return ATTN_ERR_ALIGN;
  c->k = static_cast<uint16_t*>(a->k);
  c->v = static_cast<uint16_t*>(a->v);
  c->weights = a->weights;
  c->positions = a->positions;
  c->table = a->block_table;
  c->lens = a->seq_lens;
  c->n_pages = a->n_pages;
  c->page_size = a->page_size;
  c->max_blocks = a->max_blocks;
  c->n_seq = a->n_seq;
  c->hkv = a->num_kv_heads;
  c->d = a->d;
  c->cap = a->max_blocks * a->page_size;
  return ATTN_OK;
}

// The new tokens' fields: offsets, and the query heads where `with_q`.
int check_tokens(const attn_new_tokens* x, bool with_q, CacheParams* c) {
  if (x == nullptr) return ATTN_ERR_NULL;
  if (x->struct_size < sizeof(attn_new_tokens)) return ATTN_ERR_CACHE;
  if (x->cu_seqlens == nullptr || (with_q && x->q == nullptr)) return ATTN_ERR_NULL;
  if (x->total < 1 || (with_q && (x->max_seqlen < 1 || x->H < 1))) return ATTN_ERR_SHAPE;
  if (with_q && (x->H % c->hkv != 0 || x->H / c->hkv > 128)) return ATTN_ERR_CACHE;
  if (!aligned(x->cu_seqlens, 4) || (with_q && !aligned(x->q, 16))) return ATTN_ERR_ALIGN;
  c->cu = x->cu_seqlens;
  c->total = x->total;
  if (with_q) {
    c->max_new = x->max_seqlen < x->total ? x->max_seqlen : x->total;
    c->group = x->H / c->hkv;
  }
  return ATTN_OK;
}

// Key rows of one copy: the largest power of two in page_size, at most 64, so
// that a copy stays within a page and a block of 128 keys is whole copies.
int piece_of(int page_size) {
  const int low = page_size & -page_size;
  return low < 64 ? low : 64;
}

int encode_pages(CUtensorMap* m, const void* ptr, const CacheParams& c, const long long st[3], int piece) {
  const long long dims[4] = {c.d, c.hkv, c.page_size, c.n_pages}, strides[3] = {st[2], st[1], st[0]};
  const int box[4] = {64, 1, piece, 1};
  return attn::encode_bf16_4d(m, ptr, dims, strides, box);
}

// q as (d, head of the group, key head, token).
int encode_queries(CUtensorMap* m, const attn_new_tokens* x, const CacheParams& c, const long long st[2], int nt) {
  const long long dims[4] = {c.d, c.group, c.hkv, c.total}, strides[3] = {st[1], st[1] * c.group, st[0]};
  const int box[4] = {64, c.group, 1, nt};
  return attn::encode_bf16_4d(m, x->q, dims, strides, box);
}

int check_scale(float scale) { return std::isfinite(scale) && scale > 0.f ? ATTN_OK : ATTN_ERR_SCALE; }

// The options that apply: the wait limit and the withheld copies of the tests.
int check_options(const attn_options* o, uint64_t* timeout_ns, unsigned int* flags) {
  unsigned int ms = kDefaultTimeoutMs;
  *flags = 0;
  if (o != nullptr) {
    if (o->struct_size < sizeof(attn_options) || o->rescale_threshold != 0.f || o->poly_exp2_mask != 0u ||
        o->counters != nullptr || (o->test_flags & ~ATTN_TEST_WITHHOLD_KV) != 0)
      return ATTN_ERR_OPTION;
    if (o->timeout_ms != 0) ms = o->timeout_ms;
    *flags = o->test_flags;
  }
  *timeout_ns = static_cast<uint64_t>(ms) * 1000000ull;
  return ATTN_OK;
}

int fail(cudaError_t e, const char* what) { return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e, what); }

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Tokens of a row tile: as many whole ones as 128 rows hold.
int tile_tokens(int group, int max_new) {
  const int nt = 128 / group;
  return nt < max_new ? nt : max_new;
}

// The attention kernel's row tiles, and its workspace: the sequences' table, then a
// part (maximum and sum, output) for each end of each CTA's range.  One row more than a
// tile holds halves the CTAs, so more tokens may need less (`bytes`); `most` is what any
// number of tokens up to max_new needs.
struct Tiles {
  int nt, per_cta, ntt, rows, max_ctas;
  size_t ml, o, bytes, most;
};
Tiles tiles_of(int group, int max_new, int d) {
  Tiles t;
  t.nt = tile_tokens(group, max_new);
  t.per_cta = t.nt < max_new ? 2 : 1;
  t.ntt = t.per_cta * t.nt < max_new ? t.per_cta * t.nt : max_new;
  t.rows = t.ntt * group;
  t.max_ctas = attn::kCacheMaxCtas / t.per_cta;
  t.ml = up256((attn::kCacheMaxSeq + 1) * sizeof(int));
  t.o = t.ml + up256(2ull * t.max_ctas * t.rows * sizeof(float2));
  t.bytes = t.o + 2ull * t.max_ctas * t.rows * d * sizeof(float);
  // With two tiles a CTA 2·160 ends of at most 2·nt·group rows: no more than one full tile's
  // 2·320 ends of nt·group.
  t.most = t.per_cta == 2 ? tiles_of(group, t.nt, d).bytes : t.bytes;
  return t;
}

// A cache of E4M3 codes and its scales.
int check_fp8(const attn_cache* a, const void* k_scales, const void* v_scales, CacheParams* c, attn::Fp8Pages* f) {
  const int rc = check_cache(a, 3, c, 16);
  if (rc != ATTN_OK) return rc;
  if (k_scales == nullptr || v_scales == nullptr || c->lens == nullptr) return ATTN_ERR_NULL;
  // (its addresses and strides count bytes: `f` has the addresses)
  f->k = static_cast<uint8_t*>(a->k);
  f->v = static_cast<uint8_t*>(a->v);
  f->ks = static_cast<uint8_t*>(const_cast<void*>(k_scales));
  f->vs = static_cast<uint8_t*>(const_cast<void*>(v_scales));
  f->per = c->page_size / attn::kFp8Block;
  c->k = c->v = nullptr;
  return ATTN_OK;
}

// The 8-bit cache's attention: the kernel for many rows or few, rows of a tile, key heads that
// a CTA works on at a time, and the workspace as above.  `most` is what any number of
// tokens up to max_new needs, of any number of sequences.
// More rows go to the converting kernel.  64 sequences of up to 8191: at d = 128 64 rows take 235 us
// there and 396 in two tiles here, 32 rows 225 and 224, but over 2000 and 100 keys 83 and 59 us and 84
// and 72, over one sequence of 32768 32 and 39; at d = 64 32 rows take 154 us and 121.
constexpr int few_rows(int d) { return d == 128 ? 16 : 32; }
struct Fp8Tiles {
  bool wide;
  int rows, hg, nt, per_cta, max_ctas;
  size_t ml, o, bytes;
};
Fp8Tiles fp8_tiles_of(int rows, int hg, int max_ctas, int d) {
  Fp8Tiles t = {false, rows, hg, 0, 1, max_ctas, 0, 0, 0};
  const size_t ends = 2ull * max_ctas * rows * hg;
  t.ml = up256((attn::kCacheMaxSeq + 1) * sizeof(int));
  t.o = t.ml + up256(ends * sizeof(float2));
  t.bytes = t.o + ends * d * sizeof(float);
  return t;
}
Fp8Tiles fp8_tiles(int group, int max_new, int d, int hg) {
  const long long all = static_cast<long long>(group) * max_new;
  if (all <= 8) return fp8_tiles_of(8, hg, attn::kCacheMaxCtas, d);  // two ranges a CTA, if apart
  if (all <= few_rows(d)) return fp8_tiles_of(all <= 16 ? 16 : 32, hg, attn::kCacheMaxCtas / 2, d);
  // As many tiles as 128 rows make, of about as many tokens each.
  const int most = tile_tokens(group, max_new), tiles = (max_new + most - 1) / most, nt = (max_new + tiles - 1) / tiles;
  const int per_cta = tiles > 1 ? 2 : 1;
  Fp8Tiles t = fp8_tiles_of(per_cta * nt * group, 1, attn::kCacheMaxCtas / per_cta, d);
  t.wide = true;
  t.nt = nt;
  t.per_cta = per_cta;
  return t;
}
size_t fp8_workspace(int group, int max_new, int d, int hg) {
  const long long all = static_cast<long long>(group) * max_new;
  size_t most = 0;
  auto count = [&](const Fp8Tiles& t) { most = t.bytes > most ? t.bytes : most; };
  count(fp8_tiles_of(8, hg, attn::kCacheMaxCtas, d));
  if (all > 8) count(fp8_tiles_of(16, hg, attn::kCacheMaxCtas / 2, d));
  if (all > 16 && few_rows(d) > 16) count(fp8_tiles_of(32, hg, attn::kCacheMaxCtas / 2, d));
  if (all > few_rows(d)) count(fp8_tiles_of(tile_tokens(group, max_new) * group, 1, attn::kCacheMaxCtas, d));
  return most;
}

// Key heads of a run: as many as a CTA's eight warps hold, where the heads allow it; of one
// sequence alone at most 2, which leaves fewer and larger parts to join (one token over 4000,
// 8000, 16000 cached ones: 12.3, 14.0, 15.9 us instead of 15.3, 16.2, 18.1; from two sequences on
// 8 is no slower: 13.7 and 15.5 us for two of 2000, 26 and 37 us for 64 of up to 500).  Pages read in
// shorter pieces cost less than that saves at every length: 1003 tokens 10.1 us instead of 10.9, 32768
// 23.5 instead of 25.3, 131072 54.6 instead of 55.4 (d = 64: 34.8 instead of 36.3).
int heads_at_once(int hkv, int n_seq) {
  const int most = n_seq == 1 ? 2 : 8;
  int hg = 1;
  while (hg < most && hkv % (2 * hg) == 0) hg *= 2;
  return hg;
}

}  // namespace

extern "C" {

size_t attn_fwd_cache_workspace_size(int H, int num_kv_heads, int max_seqlen, int d) {
  if (H < 1 || num_kv_heads < 1 || H % num_kv_heads != 0 || H / num_kv_heads > 128 || max_seqlen < 1 ||
      max_seqlen > ATTN_CACHE_MAX_NEW || (d != 64 && d != 128))
    return 0;
  return tiles_of(H / num_kv_heads, max_seqlen, d).most;
}

int attn_fwd_cache(const attn_cache* cache, const attn_new_tokens* x, const int* parents, float scale, void* o,
                   float* lse, void* workspace, size_t workspace_bytes, const attn_options* opts,
                   cudaStream_t stream) {
  if (o == nullptr || lse == nullptr) return ATTN_ERR_NULL;
  attn::CacheAttnLaunch a;
  std::memset(&a, 0, sizeof(a));
  CacheParams& c = a.p.c;
  int rc = check_cache(cache, 3, &c);
  if (rc != ATTN_OK || (rc = check_tokens(x, true, &c)) != ATTN_OK) return rc;
  if (x->k == nullptr || x->v == nullptr || c.lens == nullptr) return ATTN_ERR_NULL;
  if (x->max_seqlen > ATTN_CACHE_MAX_NEW) return ATTN_ERR_SHAPE;
  const Tiles w = tiles_of(c.group, c.max_new, c.d);
  const long long tiles = (c.max_new + w.ntt - 1) / w.ntt;
  // Units and rows of the two kernels' grids.
  if (tiles * c.n_seq * c.hkv > kMaxInt / (c.cap / 128 + 3) || tiles * c.n_seq * c.hkv * w.rows > kMaxInt ||
      static_cast<long long>(x->H) * c.total > kMaxInt)
    return ATTN_ERR_SHAPE;
  if ((rc = check_scale(scale)) != ATTN_OK) return rc;
  const long long hd = static_cast<long long>(x->H) * c.d, kd = static_cast<long long>(c.hkv) * c.d;
  const long long q_dense[2] = {hd, c.d}, k_dense[2] = {kd, c.d};
  long long qs[2], ks[2], vs[2];
  if (!resolve<2>(x->q_strides, q_dense, qs) || !resolve<2>(x->k_strides, k_dense, ks) ||
      !resolve<2>(x->v_strides, k_dense, vs))
    return ATTN_ERR_CACHE;
  if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(parents, 4))
    return ATTN_ERR_ALIGN;
  if ((rc = check_options(opts, &a.p.timeout_ns, &a.p.test_flags)) != ATTN_OK) return rc;
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.bytes) return ATTN_ERR_WORKSPACE;
  int sms = 0;
  if ((rc = attn::usable_device(&a.device, &a.p.status, &sms)) != ATTN_OK) return rc;

  a.p.parents = parents;
  a.p.o = static_cast<uint16_t*>(o);
  a.p.lse = lse;
  char* const ws = static_cast<char*>(workspace);
  a.p.ws_table = reinterpret_cast<int*>(ws);
  a.p.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.p.ws_o = reinterpret_cast<float*>(ws + w.o);
  a.p.rows = w.rows;
  a.p.wide = w.rows > attn::kWideRows;
  a.p.hg = 1;
  a.p.nt = w.nt;
  a.p.ntt = w.ntt;
  a.tiles = w.per_cta;
  a.p.piece = piece_of(c.page_size);
  a.p.scale_log2 = scale * 1.4426950408889634f;
  const int ctas = 2 * sms / w.per_cta;
  a.grid = ctas < w.max_ctas ? ctas : w.max_ctas;
  a.stream = stream;
  const long long new_dims[4] = {c.d, c.hkv, c.total, 1};
  const int new_box[4] = {64, 1, 16, 1};
  const long long kn[3] = {ks[1], ks[0], ks[0]}, vn[3] = {vs[1], vs[0], vs[0]};
  if ((rc = encode_queries(&a.q, x, c, qs, w.nt)) != ATTN_OK || (rc = encode_pages(&a.k, c.k, c, c.k_st, a.p.piece)) != ATTN_OK ||
      (rc = encode_pages(&a.v, c.v, c, c.v_st, a.p.piece)) != ATTN_OK ||
      (rc = attn::encode_bf16_4d(&a.kn, x->k, new_dims, kn, new_box)) != ATTN_OK ||
      (rc = attn::encode_bf16_4d(&a.vn, x->v, new_dims, vn, new_box)) != ATTN_OK)
    return rc;
  return fail(attn::launch_cache_attn(a), "cache attention launch");
}

int attn_cache_append(const attn_cache* cache, const attn_new_tokens* x, const int* rows, int n_rows,
                      const int* seq_pos, cudaStream_t stream) {
  attn::CacheAppendParams p;
  std::memset(&p, 0, sizeof(p));
  int rc = check_cache(cache, 3, &p.c);
  if (rc != ATTN_OK || (rc = check_tokens(x, false, &p.c)) != ATTN_OK) return rc;
  if (x->k == nullptr || x->v == nullptr || p.c.lens == nullptr) return ATTN_ERR_NULL;
  if ((rows != nullptr && n_rows < 1) || x->total > kMaxCapacity || n_rows > kMaxCapacity) return ATTN_ERR_SHAPE;
  p.n_rows = rows != nullptr ? n_rows : x->total;
  const long long kd = static_cast<long long>(p.c.hkv) * p.c.d, dense[2] = {kd, p.c.d};
  if (!resolve<2>(x->k_strides, dense, p.kn_st) || !resolve<2>(x->v_strides, dense, p.vn_st)) return ATTN_ERR_CACHE;
  if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(rows, 4) || !aligned(seq_pos, 4)) return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  if ((rc = attn::usable_device(&dev, &status, &sms)) != ATTN_OK) return rc;
  p.kn = static_cast<const uint16_t*>(x->k);
  p.vn = static_cast<const uint16_t*>(x->v);
  p.rows = rows;
  p.seq_pos = seq_pos;
  return fail(attn::launch_cache_append(p, stream), "cache append launch");
}

int attn_cache_weights(const attn_cache* cache, const attn_new_tokens* x, const float* lse, float scale,
                       float* weights_out, const attn_options* opts, cudaStream_t stream) {
  if (lse == nullptr || weights_out == nullptr) return ATTN_ERR_NULL;
  attn::CacheWeightLaunch a;
  std::memset(&a, 0, sizeof(a));
  CacheParams& c = a.p.c;
  int rc = check_cache(cache, 1, &c);
  if (rc != ATTN_OK || (rc = check_tokens(x, true, &c)) != ATTN_OK) return rc;
  if (c.lens == nullptr) return ATTN_ERR_NULL;
  const long long tiles = static_cast<long long>(c.n_seq) * c.hkv * ((c.cap + 255) / 256);
  // (128: the kernel rounds a sequence's rows up to whole chunks)
  if (tiles > kMaxInt || static_cast<long long>(x->H) * c.total > kMaxInt - 128) return ATTN_ERR_SHAPE;
  if ((rc = check_scale(scale)) != ATTN_OK) return rc;
  if (scale < ATTN_CACHE_MIN_SCALE) return ATTN_ERR_SCALE;  // (the kernel divides the LSE by it)
  const long long dense[2] = {static_cast<long long>(x->H) * c.d, c.d};
  long long qs[2];
  if (!resolve<2>(x->q_strides, dense, qs)) return ATTN_ERR_CACHE;
  if (!aligned(lse, 4) || !aligned(weights_out, 16)) return ATTN_ERR_ALIGN;
  if ((rc = check_options(opts, &a.p.timeout_ns, &a.p.test_flags)) != ATTN_OK) return rc;
  int sms = 0;
  if ((rc = attn::usable_device(&a.device, &a.p.status, &sms)) != ATTN_OK) return rc;
  a.p.lse = lse;
  a.p.out = weights_out;
  a.p.nt = tile_tokens(c.group, c.max_new);
  a.p.n_cols = (a.p.nt * c.group + 15) & ~15;
  a.p.by_hkv = attn::fast_div(c.hkv);
  a.p.by_page = attn::fast_div(c.page_size);
  a.p.by_nt = attn::fast_div(a.p.nt);
  a.p.piece = piece_of(c.page_size);
  a.p.scale_log2 = scale * 1.4426950408889634f;
  a.p.inv_scale = 1.f / scale;
  a.tiles = static_cast<int>(tiles);
  a.grid = tiles < sms ? static_cast<int>(tiles) : sms;
  // CTAs that share a tile, where its rows make 8 chunks and more (of 4, a second CTA
  // cost more than it gave).  The tiles are known on the device only.  As many as the
  // table has room for decide on clusters of 8 and 4, which leave SMs without work if
  // there are more tiles than expected.  Clusters of 2 fill the GPU and part where the
  // tiles are many; they are launched if whole prompts of these rows make few enough.
  // The bounds are where the times in cache_weights.cu cross: 512 tiles of up to 63
  // chunks take 150 us shared by two and 185 otherwise, of up to 32 chunks 91 and 84.
  const int chunks = (c.max_new + a.p.nt - 1) / a.p.nt;
  const long long prompts = c.hkv * (c.total / 256ll + c.n_seq);
  a.p.share_most = (chunks >= 48 ? 4 : 2) * sms;
  if (chunks >= 8 && (tiles < prompts ? tiles : prompts) <= a.p.share_most)
    a.p.log_split = chunks >= 64 && 4 * tiles <= sms ? 3 : (8 * tiles <= 5ll * sms ? 2 : 1);
  a.stream = stream;
  if ((rc = encode_queries(&a.q, x, c, qs, a.p.nt)) != ATTN_OK || (rc = encode_pages(&a.k, c.k, c, c.k_st, a.p.piece)) != ATTN_OK)
    return rc;
  return fail(attn::launch_cache_weights(a), "cache weights launch");
}

int attn_cache_select(const attn_cache* cache, const int* seq_pos, int budget, int recent, int* kept,
                      cudaStream_t stream) {
  if (kept == nullptr) return ATTN_ERR_NULL;
  CacheParams c;
  int rc = check_cache(cache, 0, &c);
  if (rc != ATTN_OK) return rc;
  if (c.weights == nullptr || c.lens == nullptr || (c.positions != nullptr && seq_pos == nullptr)) return ATTN_ERR_NULL;
  if (budget < 1 || budget > kMaxCapacity || recent < 0 || recent > budget || c.cap > ATTN_CACHE_MAX_SELECT ||
      static_cast<long long>(c.n_seq) * c.hkv > kMaxInt)
    return ATTN_ERR_SHAPE;
  if (!aligned(kept, 4) || !aligned(seq_pos, 4)) return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  if ((rc = attn::usable_device(&dev, &status, &sms)) != ATTN_OK) return rc;
  return fail(attn::launch_cache_select(c, seq_pos, budget, recent, kept, dev, stream), "cache select launch");
}

int attn_cache_compact(const attn_cache* cache, const int* kept, int budget, cudaStream_t stream) {
  if (kept == nullptr) return ATTN_ERR_NULL;
  CacheParams c;
  int rc = check_cache(cache, 3, &c);
  if (rc != ATTN_OK) return rc;
  if (budget < 1 || budget > kMaxCapacity ||
      static_cast<long long>(c.n_seq) * c.hkv * ((budget + 31) / 32) > kMaxInt)
    return ATTN_ERR_SHAPE;
  if (!aligned(kept, 4)) return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  if ((rc = attn::usable_device(&dev, &status, &sms)) != ATTN_OK) return rc;
  return fail(attn::launch_cache_compact(c, kept, budget, stream), "cache compact launch");
}

size_t attn_fwd_cache_fp8_workspace_size(int H, int num_kv_heads, int max_seqlen, int d) {
  if (H < 1 || num_kv_heads < 1 || H % num_kv_heads != 0 || H / num_kv_heads > 128 || max_seqlen < 1 ||
      max_seqlen > ATTN_CACHE_MAX_NEW || (d != 64 && d != 128))
    return 0;
  return fp8_workspace(H / num_kv_heads, max_seqlen, d, heads_at_once(num_kv_heads, 2));
}

int attn_fwd_cache_fp8(const attn_cache* cache, const void* k_scales, const void* v_scales, const attn_new_tokens* x,
                       const int* parents, float scale, void* o, float* lse, void* workspace, size_t workspace_bytes,
                       const attn_options* opts, cudaStream_t stream) {
  if (o == nullptr || lse == nullptr) return ATTN_ERR_NULL;
  attn::CacheAttnFp8Launch a;
  std::memset(&a, 0, sizeof(a));
  CacheParams& c = a.p.c;
  int rc = check_fp8(cache, k_scales, v_scales, &c, &a.f);
  if (rc != ATTN_OK || (rc = check_tokens(x, true, &c)) != ATTN_OK) return rc;
  if (x->k == nullptr || x->v == nullptr) return ATTN_ERR_NULL;
  if (x->max_seqlen > ATTN_CACHE_MAX_NEW) return ATTN_ERR_SHAPE;
  const int hg = heads_at_once(c.hkv, c.n_seq);
  const Fp8Tiles w = fp8_tiles(c.group, c.max_new, c.d, hg);
  const long long tiles = (static_cast<long long>(c.group) * c.max_new + w.rows - 1) / w.rows;
  // Units and rows of the two kernels' grids.
  if (tiles * c.n_seq * c.hkv > kMaxInt / (c.cap / 128 + 3) || tiles * c.n_seq * c.hkv * w.rows > kMaxInt ||
      static_cast<long long>(x->H) * c.total > kMaxInt)
    return ATTN_ERR_SHAPE;
  if ((rc = check_scale(scale)) != ATTN_OK) return rc;
  const long long hd = static_cast<long long>(x->H) * c.d, kd = static_cast<long long>(c.hkv) * c.d;
  const long long q_dense[2] = {hd, c.d}, k_dense[2] = {kd, c.d};
  if (!resolve<2>(x->q_strides, q_dense, a.q_st) || !resolve<2>(x->k_strides, k_dense, a.kn_st) ||
      !resolve<2>(x->v_strides, k_dense, a.vn_st))
    return ATTN_ERR_CACHE;
  if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(parents, 4))
    return ATTN_ERR_ALIGN;
  if ((rc = check_options(opts, &a.p.timeout_ns, &a.p.test_flags)) != ATTN_OK) return rc;
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.bytes) return ATTN_ERR_WORKSPACE;
  int sms = 0;
  if ((rc = attn::usable_device(&a.device, &a.p.status, &sms)) != ATTN_OK) return rc;

  a.q = static_cast<const uint16_t*>(x->q);
  a.kn = static_cast<const uint16_t*>(x->k);
  a.vn = static_cast<const uint16_t*>(x->v);
  a.p.parents = parents;
  a.p.o = static_cast<uint16_t*>(o);
  a.p.lse = lse;
  char* const ws = static_cast<char*>(workspace);
  a.p.ws_table = reinterpret_cast<int*>(ws);
  a.p.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.p.ws_o = reinterpret_cast<float*>(ws + w.o);
  a.p.rows = w.rows;
  a.p.hg = w.hg;
  // Parts chunk by chunk where their tiles are many: the join of few tiles takes a row a block (one
  // sequence of 4096 and 60 tokens in 19 parts: 37 us chunk by chunk).
  a.p.wide = w.rows > attn::kWideRows && tiles * c.n_seq * c.hkv * c.d > 8ll * (2 / w.per_cta * sms);
  a.p.nt = w.nt;
  a.p.ntt = w.per_cta * w.nt;
  a.tiles = w.per_cta;
  a.p.piece = attn::kFp8Block;
  a.p.scale_log2 = scale * 1.4426950408889634f;
  const int ctas = w.wide && w.per_cta == 1 ? 2 * sms : sms;
  const int most = w.wide ? w.max_ctas : attn::kCacheMaxCtas / 2;
  a.grid = ctas < most ? ctas : most;
  // Where each CTA has eight tiles or more, most of the time is in their starts and ends, which two
  // groups of warps overlap better apart (8 key heads, d = 128: 2000 sequences of up to 50 97 us instead of
  // 111, of up to 500 261 instead of 268); fewer tiles cost more parts to join (1024 of up to 500 157
  // instead of 154, 608 112 instead of 106).
  a.apart = !w.wide && w.rows == 8 && tiles * c.n_seq * (c.hkv / hg) >= 8 * a.grid;
  a.stream = stream;
  if (w.wide) {
    if ((rc = encode_queries(&a.q_map, x, c, a.q_st, w.nt)) != ATTN_OK) return rc;
    return fail(attn::launch_cache_attn_fp8_wide(a), "8-bit cache attention launch");
  }
  return fail(attn::launch_cache_attn_fp8(a), "8-bit cache attention launch");
}

int attn_cache_append_fp8(const attn_cache* cache, void* k_scales, void* v_scales, const attn_new_tokens* x,
                          const int* rows, int n_rows, cudaStream_t stream) {
  attn::CacheAppendFp8Params p;
  std::memset(&p, 0, sizeof(p));
  int rc = check_fp8(cache, k_scales, v_scales, &p.c, &p.f);
  if (rc != ATTN_OK || (rc = check_tokens(x, false, &p.c)) != ATTN_OK) return rc;
  if (x->k == nullptr || x->v == nullptr) return ATTN_ERR_NULL;
  p.n_rows = rows != nullptr ? n_rows : x->total;
  if ((rows != nullptr && n_rows < 1) || x->total > kMaxCapacity || n_rows > kMaxCapacity ||
      (p.n_rows / 16 + 2ll * p.c.n_seq) * 2 * p.c.hkv > kMaxInt)
    return ATTN_ERR_SHAPE;
  const long long kd = static_cast<long long>(p.c.hkv) * p.c.d, dense[2] = {kd, p.c.d};
  if (!resolve<2>(x->k_strides, dense, p.kn_st) || !resolve<2>(x->v_strides, dense, p.vn_st)) return ATTN_ERR_CACHE;
  if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(rows, 4)) return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  if ((rc = attn::usable_device(&dev, &status, &sms)) != ATTN_OK) return rc;
  p.kn = static_cast<const uint16_t*>(x->k);
  p.vn = static_cast<const uint16_t*>(x->v);
  p.rows = rows;
  return fail(attn::launch_cache_append_fp8(p, stream), "8-bit cache append launch");
}

int attn_cache_gather_fp8(const attn_cache* cache, const void* k_scales, const void* v_scales, const int* cu_out,
                          int total, void* k_out, void* v_out, cudaStream_t stream) {
  if (cu_out == nullptr || k_out == nullptr || v_out == nullptr) return ATTN_ERR_NULL;
  attn::CacheGatherFp8Params p;
  std::memset(&p, 0, sizeof(p));
  int rc = check_fp8(cache, k_scales, v_scales, &p.c, &p.f);
  if (rc != ATTN_OK) return rc;
  if (total < 1 || total > kMaxCapacity) return ATTN_ERR_SHAPE;
  if (!aligned(cu_out, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  if ((rc = attn::usable_device(&dev, &status, &sms)) != ATTN_OK) return rc;
  p.c.cu = cu_out;
  p.c.total = total;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  return fail(attn::launch_cache_gather_fp8(p, stream), "8-bit cache gather launch");
}

int attn_cache_pages(const attn_pages* t, const int* seq_lens, int* missing, const int* cu_new, int total,
                     long long* slots, int* positions, cudaStream_t stream) {
  if (t == nullptr || seq_lens == nullptr || missing == nullptr) return ATTN_ERR_NULL;
  if (t->struct_size < sizeof(attn_pages)) return ATTN_ERR_CACHE;
  if (t->block_table == nullptr || t->n_blocks == nullptr || t->free_pages == nullptr || t->n_free == nullptr ||
      (cu_new != nullptr && total > 0 && (slots == nullptr || positions == nullptr)))
    return ATTN_ERR_NULL;
  if (t->n_seq < 1 || t->max_blocks < 1 || t->n_pages < 1 || total < 0 || total > kMaxCapacity ||
      static_cast<long long>(t->n_seq) * t->max_blocks > kMaxInt)
    return ATTN_ERR_SHAPE;
  if (t->page_size < 16 || t->page_size > 65536 || t->page_size % 16 != 0 || t->n_seq > attn::kCacheMaxSeq ||
      static_cast<long long>(t->max_blocks) * t->page_size > kMaxCapacity)
    return ATTN_ERR_CACHE;
  if (!aligned(t->block_table, 4) || !aligned(t->n_blocks, 4) || !aligned(t->free_pages, 4) || !aligned(t->n_free, 4) ||
      !aligned(seq_lens, 4) || !aligned(missing, 4) || !aligned(cu_new, 4) || !aligned(slots, 8) || !aligned(positions, 4))
    return ATTN_ERR_ALIGN;
  int dev = -1, sms = 0;
  unsigned int* status = nullptr;
  const int rc = attn::usable_device(&dev, &status, &sms);
  if (rc != ATTN_OK) return rc;
  attn::CachePagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.lens = seq_lens;
  p.table = t->block_table;
  p.n_blocks = t->n_blocks;
  p.free_pages = t->free_pages;
  p.n_free = t->n_free;
  p.missing = missing;
  p.cu = cu_new;
  p.slots = slots;
  p.positions = positions;
  p.n_seq = t->n_seq;
  p.max_blocks = t->max_blocks;
  p.n_pages = t->n_pages;
  p.page_size = t->page_size;
  p.total = total;
  p.by_page = attn::fast_div(t->page_size);
  return fail(attn::launch_cache_pages(p, stream), "page tables launch");
}

}  // extern "C"
