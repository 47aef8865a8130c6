// Pages of a cache's sequences: spec_tree_kv_reserve and spec_tree_kv_release.
//
// A sequence's share of the free list is a prefix sum over the sequences, which
// every CTA takes for itself over those before its own (and, to give pages back,
// over all): two words each, read from the L2, instead of a second launch.  Lengths
// and counts are written by whichever CTA is the last to have read them.  64 sequences
// take 4 us either way, 512 with 800 slots each 7 to reserve and 5 to release: a launch,
// the sum, and the last CTA's pass over what the others left.
#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_CTAS = 512;

// The sum over the CTA of each thread's two numbers.
__device__ __forceinline__ void block_sum(int64_t& a, int64_t& b) {
  __shared__ int64_t part[2][THREADS / 32];
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[0][threadIdx.x / 32] = a, part[1][threadIdx.x / 32] = b;
  __syncthreads();
  a = b = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) a += part[0][w], b += part[1][w];
}

__device__ __forceinline__ int held_by(const spec_tree_pages_t& p, int b) { return min(max(p.held[b], 0), p.max_pages); }

// Pages that sequence b lacks; `tokens`: slots that are to have pages, -1 for
// a length that none has; a need past the table counts as none.
__device__ __forceinline__ int lacking(const ReserveLaunch& L, int b, int page_shift, int64_t& tokens) {
  const int len = L.seq_len[b];
  int n = L.count;
  if (L.n_nodes) n = min(n, max(L.n_nodes[b], 0));
  tokens = len < 0 ? -1 : static_cast<int64_t>(len) + n;
  const int64_t need = (tokens + L.pages.page_size - 1) >> page_shift;
  return len < 0 || need > L.pages.max_pages ? 0 : max(static_cast<int>(need) - held_by(L.pages, b), 0);
}

// Pages that sequence b gives back, and those that it keeps.
__device__ __forceinline__ int returned(const ReleaseLaunch& L, int b, int page_shift, int& kept) {
  const int keep = L.keep[b], held = held_by(L.pages, b);
  kept = keep < 0 ? held : static_cast<int>(min64(held, (static_cast<int64_t>(keep) + L.pages.page_size - 1) >> page_shift));
  return held - kept;
}

// The last CTA to come adds the changes in scratch[1 ..] to the counts.
__device__ __forceinline__ void settle_counts(const spec_tree_pages_t& p, int B) {
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.scratch, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  int64_t sum = 0, none = 0;
  for (int b = threadIdx.x; b < B; b += THREADS) {
    const int change = __ldcg(p.scratch + 1 + b);
    p.scratch[1 + b] = 0;
    if (change) p.held[b] = held_by(p, b) + change;
    sum += change;
  }
  block_sum(sum, none);
  if (threadIdx.x == 0) {
    p.n_free[0] -= static_cast<int>(sum);
    p.scratch[0] = 0;
  }
}

__global__ void __launch_bounds__(THREADS) kv_reserve_kernel(const ReserveLaunch L, int per_cta, int page_shift) {
  const spec_tree_pages_t& p = L.pages;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b0 = blockIdx.x * per_cta, b1 = min(b0 + per_cta, L.B);
  int64_t before = 0, none = 0, tokens;
  for (int b = threadIdx.x; b < b0; b += THREADS) before += lacking(L, b, page_shift, tokens);
  block_sum(before, none);
  const int n_free = min(max(p.n_free[0], 0), p.n_pages);
  for (int b = b0; b < b1; ++b) {
    const int lack = lacking(L, b, page_shift, tokens), held = held_by(p, b);
    const bool granted = lack == 0 || before + lack <= n_free;
    const int add = granted ? lack : 0;
    // the pages before + j of the free list, from its end
    const int64_t top = n_free - 1 - before;
    int32_t* row = p.page_table + static_cast<int64_t>(b) * p.table_stride;
    for (int j = threadIdx.x; j < add; j += THREADS) row[held + j] = p.free_pages[top - j];
    if (threadIdx.x == 0) {
      p.scratch[1 + b] = add;
      if (tokens < 0) set_status(L.status, SPEC_TREE_S_NODES);
      if (!granted || tokens > static_cast<int64_t>(p.max_pages) << page_shift) set_status(L.status, SPEC_TREE_S_PAGES);
    }
    if (L.slots) {
      const int64_t first = max(L.seq_len[b], 0);
      for (int i = threadIdx.x; i < L.count; i += THREADS) {
        const int64_t slot = first + i, idx = slot >> page_shift;
        int64_t at = -1;
        if (slot < tokens && idx < held + add) {
          const int page = idx < held ? row[idx] : p.free_pages[top - (idx - held)];
          if (page >= 0 && page < p.n_pages) at = (static_cast<int64_t>(page) << page_shift) + (slot & (p.page_size - 1));
        }
        L.slots[static_cast<int64_t>(b) * L.count + i] = at;
      }
    }
    before += lack;
  }
  settle_counts(p, L.B);
}

__global__ void __launch_bounds__(THREADS) kv_release_kernel(const ReleaseLaunch L, int per_cta, int page_shift) {
  const spec_tree_pages_t& p = L.pages;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b0 = blockIdx.x * per_cta, b1 = min(b0 + per_cta, L.B);
  int64_t before = 0, total = 0;
  int kept;
  for (int b = threadIdx.x; b < L.B; b += THREADS) {
    const int back = returned(L, b, page_shift, kept);
    total += back;
    if (b < b0) before += back;
  }
  block_sum(before, total);
  const int n_free = min(max(p.n_free[0], 0), p.n_pages);
  const bool room = n_free + total <= p.n_pages;
  for (int b = b0; b < b1; ++b) {
    const int back = returned(L, b, page_shift, kept);
    const int64_t top = n_free + total - 1 - before;
    int32_t* row = p.page_table + static_cast<int64_t>(b) * p.table_stride;
    for (int j = threadIdx.x; room && j < back; j += THREADS) {
      p.free_pages[top - j] = row[kept + j];
      row[kept + j] = -1;
    }
    if (threadIdx.x == 0) {
      p.scratch[1 + b] = room ? -back : 0;
      if (L.keep[b] < 0) set_status(L.status, SPEC_TREE_S_NODES);
    }
    before += back;
  }
  if (!room && blockIdx.x == 0 && threadIdx.x == 0) set_status(L.status, SPEC_TREE_S_PAGES);
  settle_counts(p, L.B);
}

// Sequences of a CTA, one after the other.
int sequences_per_cta(int B) { return (B + MAX_CTAS - 1) / MAX_CTAS; }

}  // namespace

cudaError_t launch_kv_reserve(const ReserveLaunch& L, cudaStream_t stream) {
  const int per = sequences_per_cta(L.B);
  return launch_pdl(kv_reserve_kernel, dim3((L.B + per - 1) / per), dim3(THREADS), 0, stream, L, per,
                    log2_of(L.pages.page_size));
}

cudaError_t launch_kv_release(const ReleaseLaunch& L, cudaStream_t stream) {
  const int per = sequences_per_cta(L.B);
  return launch_pdl(kv_release_kernel, dim3((L.B + per - 1) / per), dim3(THREADS), 0, stream, L, per,
                    log2_of(L.pages.page_size));
}

}  // namespace st
