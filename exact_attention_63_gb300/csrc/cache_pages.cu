// Block tables from the requests' lengths, and the slots of their new tokens.
//
// A cluster of CTAs resizes the tables: with want = ⌈len / page_size⌉, first every sequence
// gives back the pages behind `want` (prefix sums over the sequences give each its place on the
// stack of free pages), then, in the sequences' order, those that want more take them from
// its top if the stack holds what they and the ones before them lack.  Every CTA makes the
// prefix sums for itself from the same counts; the pages that change hands are dealt out to
// all of their warps, whoever they belong to.  Latency bounds it: two prefix sums over up to 2048
// sequences, and the chain length → sum → stack → table.  (24,500 pages: 9 us, 24 by one CTA of 1024
// threads.)  Calls that place few tokens are one CTA's (below).
#include "attn_gb300.h"
#include "cache_device.cuh"

namespace attn {
namespace {

constexpr int kPagesThreads = 512, kPagesCtas = 8;
constexpr int kFewTokens = 4096;  // slots of so many tokens are written by the same CTAs

// get(s, i), then put(s, i, what it got), for all i in [0, count) with tab[s] <= i < tab[s + 1]:
// a warp has a run of the numbers, 32 lanes side by side and four steps at once.  (Unsigned: up to
// 2^31 - 1 of them are rounded up to the warps' runs.)
template <class G, class P>
__device__ __forceinline__ void deal_out(const int* tab, int n, int count, G get, P put) {
  const unsigned int lane = threadIdx.x & 31, warps = gridDim.x * (kPagesThreads / 32);
  const unsigned int warp = blockIdx.x * (kPagesThreads / 32) + (threadIdx.x >> 5);
  const unsigned int per = ((count + warps - 1) / warps + 31) & ~31u;
  const unsigned int end = min(static_cast<unsigned int>(count), (warp + 1) * per);
  unsigned int at = warp * per;
  if (at >= end) return;
  int s = 0;
  for (; at < end; at += 128) {
    int who[4], got[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned int i = at + 32 * k + lane;
      if (i < end && tab[s + 1] <= static_cast<int>(i)) s = find_seq(tab, n, static_cast<int>(i), s);
      who[k] = s;
      if (i < end) got[k] = get(s, static_cast<int>(i));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned int i = at + 32 * k + lane;
      if (i < end) put(who[k], static_cast<int>(i), got[k]);
    }
  }
}

__device__ __forceinline__ void write_slot(const CachePagesParams& p, const int* cu, int i) {
  const int s = find_seq(cu, p.n_seq, i);
  const int a = min(max(cu[s], 0), p.total), z = min(max(cu[s + 1], a), p.total);
  if (i < a || i >= z) return;
  const int slot = p.lens[s] - z + i;
  long long at = -1;
  if (slot >= 0 && p.missing[s] == 0) {
    const int blk = p.by_page(slot);
    if (blk < p.max_blocks)
      at = static_cast<long long>(p.table[static_cast<long long>(s) * p.max_blocks + blk]) * p.page_size +
           (slot - blk * p.page_size);
  }
  p.slots[i] = at;
  p.positions[i] = slot;
}

// All CTAs of the (one) cluster; what they wrote to global memory is visible to each other.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPagesThreads) cache_pages_kernel(const CachePagesParams p, int tokens_here) {
  __shared__ int tab[kCacheMaxSeq + 1], sums[kPagesThreads / 32], s_old[kCacheMaxSeq], s_want[kCacheMaxSeq], s_grown;
  const int n = p.n_seq;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int s = threadIdx.x; s < n; s += kPagesThreads) {
    s_want[s] = p.by_page(min(max(p.lens[s], 0), 0x7FFFFFFF - p.page_size) + p.page_size - 1);
    s_old[s] = min(max(p.n_blocks[s], 0), p.max_blocks);
  }
  int top = min(max(*p.n_free, 0), p.n_pages);
  if (threadIdx.x == 0) s_grown = 0;
  __syncthreads();
  // ---- pages that go back
  prefix_table(n, tab, sums, [&](int s) { return max(s_old[s] - s_want[s], 0); });
  const int back = tab[n];
  cluster_sync();  // all have read the counts and the stack's height
  auto dropped = [&](int s, int i) { return p.table + static_cast<long long>(s) * p.max_blocks + s_want[s] + (i - tab[s]); };
  deal_out(tab, n, back, [&](int s, int i) { return *dropped(s, i); }, [&](int s, int i, int page) {
    // (a stack that is full holds them all already)
    if (top + static_cast<long long>(i) < p.n_pages) p.free_pages[top + i] = page;
    *dropped(s, i) = -1;
  });
  top = static_cast<int>(min(static_cast<long long>(top) + back, static_cast<long long>(p.n_pages)));
  cluster_sync();
  // ---- pages that are taken: tab counts what is wanted, served or not
  prefix_table(n, tab, sums, [&](int s) {
    return s_want[s] <= p.max_blocks ? max(s_want[s] - s_old[s], 0) : 0;
  });
  for (int s = threadIdx.x; s < n; s += kPagesThreads) {
    const int want = s_want[s], old = s_old[s], held = min(old, want);
    const bool wide = want > p.max_blocks, served = !wide && (want <= old || tab[s + 1] <= top);
    if (blockIdx.x == 0) {
      p.n_blocks[s] = served ? want : held;
      p.missing[s] = served ? 0 : want - held;
    }
    if (served && want > old) atomicMax(&s_grown, tab[s + 1]);  // (the served ones' needs come first)
  }
  __syncthreads();
  const int grown = s_grown;
  deal_out(tab, n, grown, [&](int, int i) { return p.free_pages[top - 1 - i]; }, [&](int s, int i, int page) {
    p.table[static_cast<long long>(s) * p.max_blocks + s_old[s] + (i - tab[s])] = page;
  });
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_free = top - grown;
  if (tokens_here == 0) return;
  cluster_sync();
  for (int s = threadIdx.x; s <= n; s += kPagesThreads) tab[s] = p.cu[s];
  __syncthreads();
  for (int i = blockIdx.x * kPagesThreads + threadIdx.x; i < tokens_here; i += gridDim.x * kPagesThreads)
    write_slot(p, tab, i);
}

// Slots and positions of many tokens, after the tables.
__global__ void __launch_bounds__(256) cache_slots_kernel(const CachePagesParams p) {
  __shared__ int cu[kCacheMaxSeq + 1];
  for (int s = threadIdx.x; s <= p.n_seq; s += 256) cu[s] = p.cu[s];
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = blockIdx.x * 1024 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = first + 256 * k;
    if (i < p.total) write_slot(p, cu, i);
  }
}

}  // namespace

cudaError_t launch_cache_pages(const CachePagesParams& p, cudaStream_t stream) {
  const bool slots = p.cu != nullptr && p.total > 0, here = slots && p.total <= kFewTokens;
  cudaError_t e;
  if (here) {
    // A decoding step, in which few pages change hands as a rule: one CTA (256 sequences, one token
    // more each: 4.3 us where a cluster takes 6.0).  A step may give back any number of pages, which
    // the host does not know.  256 requests of 4096 tokens in pages of 16, of which so many end at once, with the
    // call that makes room for them again, by one CTA and by a cluster: 4 of them 9.7 and 11.2 us, 16 (4096
    // pages) 11.2 and 11.6, half (32,768 pages) 25.7 and 14.3; 16 of 64 requests of 8191 (8192 pages) 12.2 and 11.2.
    cache_pages_kernel<<<1, kPagesThreads, 0, stream>>>(p, p.total);
    e = cudaGetLastError();
  } else {
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = kPagesCtas;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t one = {};
    one.gridDim = dim3(kPagesCtas);
    one.blockDim = dim3(kPagesThreads);
    one.stream = stream;
    one.attrs = &cluster;
    one.numAttrs = 1;
    e = cudaLaunchKernelEx(&one, cache_pages_kernel, p, 0);
  }
  if (e != cudaSuccess || !slots || here) return e;
  cudaLaunchAttribute attr;  // starts while the tables are resized, which hides its launch
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>((p.total + 1023ll) / 1024));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_slots_kernel, p);
}

}  // namespace attn
