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

// All zero → dense; else positive multiples of 8 below 2^38 (TMA: 16-byte
// multiples below 2^40 bytes).
template <int N>
bool resolve(const long long in[N], const long long dense[N], long long out[N]) {
  bool zero = true;
  for (int i = 0; i < N; ++i) zero = zero && in[i] == 0;
  for (int i = 0; i < N; ++i) {
    if (!zero && (in[i] <= 0 || (in[i] & 7) != 0 || in[i] >= (1ll << 38))) return false;
    out[i] = zero ? dense[i] : in[i];
  }
  return true;
}

// The cache's fields that every operator needs; k and v where `kv` says so
// (bit 0: k, bit 1: v).
int check_cache(const attn_cache* a, int kv, CacheParams* c) {
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
  if ((kv & 1) && !resolve<3>(a->k_strides, dense, c->k_st)) return ATTN_ERR_CACHE;
  if ((kv & 2) && !resolve<3>(a->v_strides, dense, c->v_st)) return ATTN_ERR_CACHE;
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

}  // extern "C"
