// Attention of a tree's nodes over a key-value cache in 4 bits
// (spec_tree_kv4_attend): one CTA per row, its warps over the tokens.
#include <math.h>

#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int THREADS = 128, WARPS = THREADS / 32;

template <typename T, int D>
__global__ void __launch_bounds__(THREADS) attend4_row_kernel(const AttendLaunch L, int page_shift) {
  constexpr int E = D / 32;
  __shared__ uint8_t seen[SPEC_TREE_MAX_NODES];
  __shared__ float tops[WARPS], sums[WARPS], outs[WARPS][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  grid_dependency_wait();
  grid_dependents_launch();
  const int head = blockIdx.x % L.n_q_heads, rest = blockIdx.x / L.n_q_heads;
  const int i = rest % L.nodes.count, b = rest / L.nodes.count, n = L.nodes.begin + i;
  const int kv_head = head / (L.n_q_heads / L.kv.n_kv_heads);
  T* out = static_cast<T*>(L.out.data) + b * L.out.tree_stride + i * L.out.node_stride + head * L.out.head_stride;
  int len = L.kv.seq_len[b], cnt = node_count(L.nodes, b);
  const bool past = static_cast<int64_t>(len) + cnt > (static_cast<int64_t>(L.kv.max_pages) << page_shift);
  if (len < 0 || past) {
    if (threadIdx.x == 0) set_status(L.status, len < 0 ? SPEC_TREE_S_NODES : SPEC_TREE_S_PAGES);
    cnt = 0;
  }
  if (n >= cnt) {
    if (threadIdx.x < D) out[threadIdx.x] = T(0.0f);
    return;
  }
  const int32_t* parent = L.nodes.parent ? L.nodes.parent + static_cast<int64_t>(b) * L.nodes.stride : nullptr;
  if (parent) {
    for (int x = threadIdx.x; x < SPEC_TREE_MAX_NODES; x += THREADS) seen[x] = 0;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int at = n; at >= 0;) {
        seen[at] = 1;
        const int up = parent[at];
        if (up >= at) set_status(L.status, SPEC_TREE_S_NODES);
        at = up < at ? up : -1;
      }
    __syncthreads();
  }
  const T* q = static_cast<const T*>(L.q.data) + b * L.q.tree_stride + i * L.q.node_stride + head * L.q.head_stride;
  float x[E], o[E], top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = static_cast<float>(q[lane * E + e]), o[e] = 0.0f;
  for (int t = warp; t <= len + n; t += WARPS) {
    if (parent && t >= len && !seen[t - len]) continue;
    const int64_t off = kv_slot_offset(L.kv, b, t, page_shift);
    if (off < 0 && lane == 0) set_status(L.status, SPEC_TREE_S_PAGES);
    uint32_t k = 0, v = 0;
    float2 ks = make_float2(0.0f, 0.0f), vs = ks;
    if (off >= 0) {
      const int64_t at = (L.layer * L.kv.layer_stride + off + kv_head * L.kv.head_stride + lane * E) / 2;
      const uint8_t* kb = static_cast<const uint8_t*>(L.kv.k) + at;
      const uint8_t* vb = static_cast<const uint8_t*>(L.kv.v) + at;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) k |= kb[e] << (8 * e), v |= vb[e] << (8 * e);
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const T*>(L.scales.data) + L.layer * L.scales.layer_stride +
                                                      kv_scale_offset(L.kv, L.scales, b, t, page_shift) +
                                                      kv_head * L.scales.head_stride);
      ks = Pair<T>::unpack(w.x), vs = Pair<T>::unpack(w.y);
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(x[e], fmaf(static_cast<float>((k >> (4 * e)) & 15u), ks.x, ks.y), s);
    s = warp_sum(s) * L.scale;
    const float next = s > top ? s : top;
    if (next == -INFINITY) {
      if (isnan(s)) sum = NAN;
      continue;
    }
    const float keep = expf(top - next), w = expf(s - next);
    top = next;
    sum = fmaf(sum, keep, w);
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(o[e], keep, w * fmaf(static_cast<float>((v >> (4 * e)) & 15u), vs.x, vs.y));
  }
  if (lane == 0) tops[warp] = top, sums[warp] = sum;
#pragma unroll
  for (int e = 0; e < E; ++e) outs[warp][lane * E + e] = o[e];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float all = -INFINITY, total = 0.0f, y = 0.0f;
  for (int w = 0; w < WARPS; ++w) all = fmaxf(all, tops[w]);
  for (int w = 0; w < WARPS; ++w) {
    const float f = tops[w] == -INFINITY ? 0.0f : expf(tops[w] - all);
    total += isnan(sums[w]) ? sums[w] : sums[w] * f;
    y += outs[w][threadIdx.x] * f;
  }
  out[threadIdx.x] = T(total == 0.0f ? 0.0f : y / total);
}

template <typename T, int D>
cudaError_t attend(const AttendLaunch& L, cudaStream_t stream) {
  return launch_pdl(attend4_row_kernel<T, D>, dim3(L.B * L.nodes.count * L.n_q_heads), dim3(THREADS), 0, stream, L,
                    log2_of(L.kv.page_size));
}

}  // namespace

cudaError_t launch_kv4_attend(const AttendLaunch& L, cudaStream_t stream) {
  if (L.nodes.count * (L.n_q_heads / L.kv.n_kv_heads) <= SPEC_TREE_KV4_FEW_ROWS) return launch_kv4_attend_few(L, stream);
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend<__nv_bfloat16, 128>(L, stream) : attend<__nv_bfloat16, 64>(L, stream);
  return L.kv.head_dim == 128 ? attend<__half, 128>(L, stream) : attend<__half, 64>(L, stream);
}

}  // namespace st
