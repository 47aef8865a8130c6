// Attention of a tree's nodes over a paged key-value cache (spec_tree_attend).
#include <math.h>

#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int THREADS = 128, WARPS = THREADS / 32;
constexpr int MASK_WORDS = SPEC_TREE_MAX_NODES / 32;

// One CTA per (tree, node, query head): each warp takes every fourth token the
// node sees, with a running maximum and sum; the warps' parts are joined in
// shared memory.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) attend_rows_kernel(const AttendLaunch L, int group, int page_shift) {
  constexpr int E = D / 32;  // elements per lane
  __shared__ uint32_t sees[MASK_WORDS];
  __shared__ float part_o[WARPS][D], part_m[WARPS], part_l[WARPS];
  const int64_t item = blockIdx.x;
  const int hq = static_cast<int>(item % L.n_q_heads);
  const int i = static_cast<int>(item / L.n_q_heads % L.nodes.count);
  const int b = static_cast<int>(item / L.n_q_heads / L.nodes.count);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  grid_dependency_wait();
  grid_dependents_launch();
  const int len = L.kv.seq_len[b], n = L.nodes.begin + i;
  T* out = static_cast<T*>(L.out.data) + b * L.out.tree_stride + i * L.out.node_stride + hq * L.out.head_stride;
  if (n >= node_count(L.nodes, b) || len < 0) {
    if (len < 0 && threadIdx.x == 0) set_status(L.status, SPEC_TREE_S_NODES);
    if (threadIdx.x < D) out[threadIdx.x] = T(0.0f);
    return;
  }
  if (L.nodes.parent && threadIdx.x < 32) {
    if (lane < MASK_WORDS) sees[lane] = 0;
    __syncwarp();
    if (lane == 0) {
      int at = n;
      while (at >= 0) {
        sees[at / 32] |= 1u << (at % 32);
        const int up = L.nodes.parent[static_cast<int64_t>(b) * L.nodes.stride + at];
        if (up >= at) {
          set_status(L.status, SPEC_TREE_S_NODES);
          break;
        }
        at = up;
      }
    }
  }
  __syncthreads();
  const T* q = static_cast<const T*>(L.q.data) + b * L.q.tree_stride + i * L.q.node_stride + hq * L.q.head_stride;
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = static_cast<float>(q[lane * E + e]) * L.scale;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int64_t base = L.layer * L.kv.layer_stride + static_cast<int64_t>(hq / group) * L.kv.head_stride + lane * E;
  for (int64_t t = warp; t <= static_cast<int64_t>(len) + n; t += WARPS) {
    const int node = static_cast<int>(t - len);
    if (node >= 0 && L.nodes.parent && !((sees[node / 32] >> (node % 32)) & 1)) continue;
    const int64_t off = kv_slot_offset(L.kv, b, t, page_shift);
    if (off < 0 && lane == 0) set_status(L.status, SPEC_TREE_S_PAGES);
    const T* k = static_cast<const T*>(L.kv.k) + base + off;
    const T* v = static_cast<const T*>(L.kv.v) + base + off;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += off < 0 ? 0.0f : qv[e] * static_cast<float>(k[e]);
    s = warp_sum(s);
    const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.0f : top;
    const float keep = expf(m - ref), w = expf(s - ref);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + (off < 0 ? 0.0f : w * static_cast<float>(v[e]));
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part_o[warp][lane * E + e] = o[e];
  if (lane == 0) part_m[warp] = m, part_l[warp] = l;
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, part_m[w]);
    const float ref = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < WARPS; ++w) {
      const float f = expf(part_m[w] - ref);
      sum += part_l[w] * f;
      acc += part_o[w][threadIdx.x] * f;
    }
    out[threadIdx.x] = T(sum == 0.0f ? 0.0f : acc / sum);
  }
}

template <typename T, int D>
cudaError_t attend(const AttendLaunch& L, cudaStream_t stream) {
  const int64_t ctas = static_cast<int64_t>(L.B) * L.nodes.count * L.n_q_heads;
  return launch_pdl(attend_rows_kernel<T, D>, dim3(static_cast<unsigned>(ctas)), dim3(THREADS), 0, stream, L,
                    L.n_q_heads / L.kv.n_kv_heads, log2_of(L.kv.page_size));
}

}  // namespace

size_t attend_workspace_bytes(int num_sms, int64_t rows, int head_dim) { return 16; }

cudaError_t launch_attend(const AttendLaunch& L, cudaStream_t stream) {
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend<__nv_bfloat16, 128>(L, stream) : attend<__nv_bfloat16, 64>(L, stream);
  return L.kv.head_dim == 128 ? attend<__half, 128>(L, stream) : attend<__half, 64>(L, stream);
}

}  // namespace st
