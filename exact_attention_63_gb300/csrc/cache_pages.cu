// Block tables from the requests' lengths, and the slots of their new tokens.
//
// One CTA resizes the tables: with want = ⌈len / page_size⌉, first every sequence gives
// back the pages behind `want` (prefix sums over the sequences give each its place on the
// stack of free pages), then, in the sequences' order, those that want more take them from
// its top if the stack holds what they and the ones before them lack.  The pages that
// change hands are dealt out to the threads one by one, whoever they belong to, so one
// long prompt takes as long as many short ones.  Latency bounds it: two prefix sums over up
// to 2048 sequences, and the chain length → sum → stack → table.
#include "attn_gb300.h"
#include "cache_device.cuh"

namespace attn {
namespace {

constexpr int kPagesThreads = 1024;
constexpr int kFewTokens = 4 * kPagesThreads;  // slots of so many tokens are written by the same CTA

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

__global__ void __launch_bounds__(kPagesThreads) cache_pages_kernel(const CachePagesParams p, int tokens_here) {
  __shared__ int tab[kCacheMaxSeq + 1], sums[32], s_old[kCacheMaxSeq], s_want[kCacheMaxSeq], s_grown;
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
  for (int i = threadIdx.x; i < back; i += kPagesThreads) {
    const int s = find_seq(tab, n, i);
    int* const entry = p.table + static_cast<long long>(s) * p.max_blocks + s_want[s] + (i - tab[s]);
    if (top + static_cast<long long>(i) < p.n_pages) p.free_pages[top + i] = *entry;  // (a stack that is full holds them all already)
    *entry = -1;
  }
  top = static_cast<int>(min(static_cast<long long>(top) + back, static_cast<long long>(p.n_pages)));
  __syncthreads();
  // ---- pages that are taken: tab counts what is wanted, served or not
  prefix_table(n, tab, sums, [&](int s) {
    return s_want[s] <= p.max_blocks ? max(s_want[s] - s_old[s], 0) : 0;
  });
  for (int s = threadIdx.x; s < n; s += kPagesThreads) {
    const int want = s_want[s], old = s_old[s], held = min(old, want);
    const bool wide = want > p.max_blocks, served = !wide && (want <= old || tab[s + 1] <= top);
    if (p.n_blocks[s] != (served ? want : held)) p.n_blocks[s] = served ? want : held;
    p.missing[s] = served ? 0 : want - held;
    if (served && want > old) atomicMax(&s_grown, tab[s + 1]);  // (the served ones' needs come first)
  }
  __syncthreads();
  const int grown = s_grown;
  for (int i = threadIdx.x; i < grown; i += kPagesThreads) {
    const int s = find_seq(tab, n, i);
    p.table[static_cast<long long>(s) * p.max_blocks + s_old[s] + (i - tab[s])] = p.free_pages[top - 1 - i];
  }
  if (threadIdx.x == 0) *p.n_free = top - grown;
  if (tokens_here == 0) return;
  __syncthreads();
  for (int s = threadIdx.x; s <= n; s += kPagesThreads) tab[s] = p.cu[s];
  __syncthreads();
  for (int i = threadIdx.x; i < tokens_here; i += kPagesThreads) write_slot(p, tab, i);
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
  cache_pages_kernel<<<1, kPagesThreads, 0, stream>>>(p, here ? p.total : 0);
  const cudaError_t e = cudaGetLastError();
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
