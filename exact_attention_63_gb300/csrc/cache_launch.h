// Internal interface between the cache operators' host code (cache_api.cu) and
// their kernels.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

constexpr int kWideRows = 64;        // parts of more rows may lie chunk by chunk
constexpr int kCacheMaxSeq = 2048;   // sequences of one call: their offsets are kept in shared memory
constexpr int kCacheMaxCtas = 320;   // row tiles at work at a time (two per SM); sizes the attention's workspace

// Division by a number fixed for the launch, as a multiplication (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994): x / d = x·mul >> (31 + log),
// exact for 0 ≤ x < 2^31 with mul = ⌈2^(31 + log) / d⌉ < 2^32, log = ⌈log2 d⌉: mul·d exceeds
// 2^(31 + log) by less than d ≤ 2^log, so x·mul/2^(31 + log) exceeds x/d by less than 1/d.
// The loaders of short tiles do several divisions a tile, one warp alone: it showed in their time.
struct FastDiv {
  unsigned int mul;
  int shift, d;
  __host__ __device__ int operator()(int x) const {
    return d == 1 ? x : static_cast<int>((static_cast<unsigned long long>(x) * mul) >> shift);
  }
};
inline FastDiv fast_div(int d) {
  int log = 0;
  while ((1ll << log) < d) ++log;
  const unsigned long long num = 1ull << (31 + log);
  return {d == 1 ? 0u : static_cast<unsigned int>((num + d - 1) / d), 31 + log, d};
}

// What every cache kernel knows of the cache and the new tokens.
struct CacheParams {
  uint16_t* k;
  uint16_t* v;
  long long k_st[3], v_st[3];  // element strides: page, slot, head
  float* weights;
  int* positions;
  const int* table;      // [n_seq, max_blocks]
  const int* lens;       // [n_seq]
  int n_pages, page_size, max_blocks, n_seq, hkv, d;
  int cap;               // max_blocks * page_size
  const int* cu;         // [n_seq + 1]
  int total, max_new, group;  // rows, most new tokens of a sequence, query heads per key head
};

struct CacheAttnParams {
  CacheParams c;
  const int* parents;
  uint16_t* o;           // [total, H, d]
  float* lse;            // [H, total]
  int* ws_table;         // [n_seq + 1] first unit of each sequence
  float2* ws_ml;         // [2 * grid, rows] running maximum (log2) and sum of a part
  float* ws_o;           // [2 * grid, rows, d] its unnormalised output
  int rows;              // row pitch of the parts
  int hg;                // key heads that a CTA works on at a time
  bool wide;             // parts lie chunk by chunk, [d/4][rows][4]
  int nt;                // tokens of a row tile: nt * group <= 128 rows
  int ntt;               // tokens of a CTA's row tiles
  int piece;             // key rows of one copy: the largest power of two in page_size, at most 64
  float scale_log2;
  unsigned int* status;
  uint64_t timeout_ns;
  unsigned int test_flags;
};

struct CacheAttnLaunch {
  CUtensorMap q, k, v, kn, vn;  // q box (64, group, 1, nt); cache box (64, 1, piece, 1); new keys box (64, 1, 16, 1)
  CacheAttnParams p;
  int tiles;             // row tiles of a CTA: 2 where a sequence may have more than 128 rows
  int grid, device;
  cudaStream_t stream;
};
cudaError_t launch_cache_attn(const CacheAttnLaunch& a);

struct CacheWeightParams {
  CacheParams c;
  const float* lse;      // [H, total]
  float* out;
  FastDiv by_hkv, by_page, by_nt;
  int nt;                // tokens of a chunk
  int n_cols;            // its rows rounded up to the MMA's multiple of 16
  int k_stages, q_stages;  // key slots of a half, chunk slots (set by the launch)
  int piece;
  int log_split;         // 2^log_split CTAs share a tile,
  int share_most;        // if there are no more tiles than these
  float scale_log2, inv_scale;
  unsigned int* status;
  uint64_t timeout_ns;
  unsigned int test_flags;
};
struct CacheWeightLaunch {
  CUtensorMap q, k;
  CacheWeightParams p;
  int tiles;             // at most, by the table's capacity
  int grid, device;      // grid: of CTAs that share no tiles
  cudaStream_t stream;
};
cudaError_t launch_cache_weights(const CacheWeightLaunch& a);

// A cache of E4M3 codes: k and v of CacheParams are null, its strides count bytes.
constexpr int kFp8Block = 16;              // slots that share a scale
constexpr int kFp8Lowest = 127 - 117, kFp8Highest = 127 + 119;  // exponent bytes of a scale
struct Fp8Pages {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;           // [n_pages, hkv, per] exponent bytes: 2^(byte - 127)
  uint8_t* vs;
  int per;               // page_size / 16
};

struct CacheAttnFp8Launch {
  CUtensorMap q_map;     // many rows: box (64, group, 1, nt)
  CacheAttnParams p;
  Fp8Pages f;
  const uint16_t* q;
  const uint16_t* kn;
  const uint16_t* vn;
  long long q_st[2], kn_st[2], vn_st[2];  // element strides: token, head
  int tiles;             // many rows: row tiles of a CTA, 2 where a sequence may have more than 128 rows
  bool apart;            // up to 8 rows: the two groups of warps of a CTA work on ranges of their own
  int grid, device;
  cudaStream_t stream;
};
cudaError_t launch_cache_attn_fp8(const CacheAttnFp8Launch& a);
cudaError_t launch_cache_attn_fp8_wide(const CacheAttnFp8Launch& a);

struct CacheAppendFp8Params {
  CacheParams c;
  Fp8Pages f;
  const uint16_t* kn;
  const uint16_t* vn;
  long long kn_st[2], vn_st[2];
  const int* rows;       // may be null
  int n_rows;            // tokens to place: entries of rows, or total
};
cudaError_t launch_cache_append_fp8(const CacheAppendFp8Params& p, cudaStream_t stream);

struct CacheGatherFp8Params {
  CacheParams c;         // cu, total: of the rows that are written
  Fp8Pages f;
  uint16_t* k_out;       // [total, hkv, d]
  uint16_t* v_out;
};
cudaError_t launch_cache_gather_fp8(const CacheGatherFp8Params& p, cudaStream_t stream);

struct CachePagesParams {
  const int* lens;       // [n_seq]
  int* table;            // [n_seq, max_blocks]
  int* n_blocks;         // [n_seq]
  int* free_pages;       // [n_pages]
  int* n_free;           // [1]
  int* missing;          // [n_seq]
  const int* cu;         // [n_seq + 1], may be null
  long long* slots;      // [total]
  int* positions;        // [total]
  int n_seq, max_blocks, n_pages, page_size, total;
  FastDiv by_page;
};
cudaError_t launch_cache_pages(const CachePagesParams& p, cudaStream_t stream);

struct CacheAppendParams {
  CacheParams c;
  const uint16_t* kn;
  const uint16_t* vn;
  long long kn_st[2], vn_st[2];
  const int* rows;       // may be null
  int n_rows;            // tokens to place: entries of rows, or total
  const int* seq_pos;
};
cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t stream);
cudaError_t launch_cache_select(const CacheParams& c, const int* seq_pos, int budget, int recent, int* kept,
                                int device, cudaStream_t stream);
cudaError_t launch_cache_compact(const CacheParams& c, const int* kept, int budget, cudaStream_t stream);

}  // namespace attn
