// Device helpers shared by the cache kernels: a sequence's new tokens and
// length (clamped to the tensors, so that a malformed table cannot lead outside
// them) and the prefix table over the sequences.
#pragma once

#include "attn_device.cuh"
#include "cache_launch.h"

namespace attn {

struct SeqRows {
  int q0, n;  // first packed row and number of rows of a sequence
};
__device__ __forceinline__ SeqRows seq_rows(const CacheParams& c, int s) {
  const int a = min(max(c.cu[s], 0), c.total), z = min(max(c.cu[s + 1], a), c.total);
  return {a, z - a};
}
__device__ __forceinline__ int seq_len(const CacheParams& c, int s) { return min(max(c.lens[s], 0), c.cap); }

// Page of slot j of sequence s, for reading: always inside the cache.
__device__ __forceinline__ int page_for_read(const CacheParams& c, int s, int block) {
  const int p = c.table[static_cast<long long>(s) * c.max_blocks + block];
  return min(max(p, 0), c.n_pages - 1);
}

// tab[s] = sum of units(0) .. units(s - 1) for s in [0, n]; every thread of the
// CTA calls it (it synchronises).  `sums`: one int per warp.
template <class F>
__device__ __forceinline__ void prefix_table(int n, int* tab, int* sums, F units) {
  const int nth = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 31, warp = tid >> 5;
  const int per = (n + nth - 1) / nth, s0 = min(n, tid * per), s1 = min(n, s0 + per);
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int u = units(s);
    tab[s + 1] = u;
    mine += u;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = incl - mine;
  for (int w = 0; w < warp; ++w) before += sums[w];
  for (int s = s0; s < s1; ++s) {
    before += tab[s + 1];
    tab[s + 1] = before;
  }
  if (tid == 0) tab[0] = 0;
  __syncthreads();
}

// The sequence s with tab[s] <= u < tab[s + 1]; `lo`: one known not to be behind it.
__device__ __forceinline__ int find_seq(const int* tab, int n, int u, int lo = 0) {
  int hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace attn
