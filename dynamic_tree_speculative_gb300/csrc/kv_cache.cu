// The paged key-value cache's writes: appending a tree's nodes with the head
// norms and the rotation on the way (spec_tree_kv_append), and moving the
// accepted path behind the committed tokens (spec_tree_kv_commit).
#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int APPEND_THREADS = 256;
constexpr int COMMIT_THREADS = 128;
constexpr int COMMIT_BATCH = 8;  // path steps loaded before any is stored

// A head vector belongs to D / 8 neighbouring lanes, 8 elements (16 bytes)
// each; a CTA takes 256 * 8 / D vectors of one node.  Everything is read and
// written once: bytes bound it, at few nodes the chain of dependent loads
// (length, position, rotation row) does.
template <typename T, int D>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const AppendLaunch L, int chunks, int page_shift) {
  constexpr int LANES = D / 8, PER_CTA = APPEND_THREADS / LANES;
  const int64_t item = blockIdx.x / chunks;
  const int b = static_cast<int>(item / L.nodes.count), i = static_cast<int>(item % L.nodes.count);
  const int head = (blockIdx.x % chunks) * PER_CTA + threadIdx.x / LANES;
  const int lane = threadIdx.x % LANES;
  const int n_kv = L.kv.n_kv_heads;
  const bool is_q = head < L.n_q_heads, is_k = !is_q && head < L.n_q_heads + n_kv;
  const bool any = head < L.n_q_heads + 2 * n_kv;
  const int h = is_q ? head : (is_k ? head - L.n_q_heads : head - L.n_q_heads - n_kv);
  grid_dependency_wait();
  grid_dependents_launch();

  const spec_tree_heads_t& in = is_q ? L.q : (is_k ? L.k : L.v);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (any)
    raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(in.data) + b * in.tree_stride + i * in.node_stride +
                                          h * in.head_stride + lane * 8);
  T* q_to = static_cast<T*>(L.q_out.data) + b * L.q_out.tree_stride + i * L.q_out.node_stride +
            (is_q ? h : 0) * L.q_out.head_stride + lane * 8;
  const int n = L.nodes.begin + i;
  const int len = L.kv.seq_len[b];
  if (n >= node_count(L.nodes, b) || len < 0) {  // uniform over the CTA
    if (len < 0 && threadIdx.x == 0) set_status(L.status, SPEC_TREE_S_NODES);
    if (any && is_q) *reinterpret_cast<uint4*>(q_to) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int depth = L.nodes.depth ? L.nodes.depth[static_cast<int64_t>(b) * L.nodes.stride + n] : n;
  const int64_t pos = static_cast<int64_t>(len) + depth;
  const int64_t off = kv_slot_offset(L.kv, b, static_cast<int64_t>(len) + n, page_shift);
  const bool has_angle = L.rot_dim > 0 && depth >= 0 && pos < L.rope_rows;
  if (L.rot_dim > 0 && !has_angle && threadIdx.x == 0) set_status(L.status, SPEC_TREE_S_NODES);

  float x[8];
  unpack8<T>(raw, x);
  const void* weight = is_q ? L.q_weight : (is_k ? L.k_weight : nullptr);
  // shuffles are executed by the whole warp, whichever heads its lanes hold
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
  if (weight) {
    const float r = rsqrtf(ss * (1.0f / D) + L.eps);
    float w[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + lane * 8), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
  }
  if (has_angle) {  // uniform over the CTA
    const float* row = L.rope + pos * L.rot_dim;
    const bool turns = lane * 8 < L.rot_dim;
    if (L.interleaved) {
      if (turns && any && (is_q || is_k)) {
        const float4 c = *reinterpret_cast<const float4*>(row + lane * 4);
        const float4 s = *reinterpret_cast<const float4*>(row + L.rot_dim / 2 + lane * 4);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[2 * e], d = x[2 * e + 1];
          x[2 * e] = a * cc[e] - d * ss4[e];
          x[2 * e + 1] = a * ss4[e] + d * cc[e];
        }
      }
    } else {
      const int half = L.rot_dim / 16;  // lanes of a half of the pairs
      const bool first = lane < half;
      const int partner = turns ? (first ? lane + half : lane - half) : lane;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(FULL, x[e], partner, LANES);
      if (turns && any && (is_q || is_k)) {
        const float* cp = row + (first ? lane : lane - half) * 8;
        const float* sp = cp + L.rot_dim / 2;
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
          const float4 c = *reinterpret_cast<const float4*>(cp + q4 * 4);
          const float4 s = *reinterpret_cast<const float4*>(sp + q4 * 4);
          const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = q4 * 4 + e;
            x[j] = first ? x[j] * cc[e] - y[j] * sn[e] : y[j] * sn[e] + x[j] * cc[e];
          }
        }
      }
    }
  }
  if (!any) return;
  if (is_q) {
    *reinterpret_cast<uint4*>(q_to) = pack8<T>(x);
    return;
  }
  if (off < 0) {
    if (lane == 0) set_status(L.status, SPEC_TREE_S_PAGES);
    return;
  }
  T* to = static_cast<T*>(is_k ? L.kv.k : L.kv.v) + L.layer * L.kv.layer_stride + off + h * L.kv.head_stride + lane * 8;
  *reinterpret_cast<uint4*>(to) = is_k ? pack8<T>(x) : raw;
}

// One thread per 16 bytes of a slot's entries in one layer of keys or values;
// it walks the path in ascending order, COMMIT_BATCH steps at a time, loading
// a batch before storing it.  Step j reads slot path[j] >= j, which only a
// step after j may write, so no entry is overwritten before it is read.
__global__ void __launch_bounds__(COMMIT_THREADS) kv_commit_kernel(const CommitLaunch L, int64_t lanes, int vecs,
                                                                   int page_shift) {
  __shared__ int64_t src[256], dst[256];
  __shared__ int bad;
  const int b = blockIdx.y;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();
  const int len = L.kv.seq_len[b];
  const int a = L.accept_len[b];
  const bool ok = len >= 0 && a >= 0 && a <= L.path_stride;
  for (int j = threadIdx.x; ok && j < a; j += COMMIT_THREADS) {
    const int node = L.out_node[static_cast<int64_t>(b) * L.path_stride + j];
    if (node <= j) {
      bad = 1;
    } else {
      src[j] = kv_slot_offset(L.kv, b, static_cast<int64_t>(len) + node, page_shift);
      dst[j] = kv_slot_offset(L.kv, b, static_cast<int64_t>(len) + j + 1, page_shift);
      if (src[j] < 0 || dst[j] < 0) {
        src[j] = dst[j] = -1;
        set_status(L.status, SPEC_TREE_S_PAGES);
      }
    }
  }
  __syncthreads();
  const bool valid = ok && !bad;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!valid) set_status(L.status, SPEC_TREE_S_NODES);
    L.new_len[b] = valid ? len + 1 + a : len;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * COMMIT_THREADS + threadIdx.x;
  if (!valid || t >= lanes) return;
  const int vec = static_cast<int>(t % vecs);
  const int64_t rest = t / vecs;
  const int h = static_cast<int>(rest % L.kv.n_kv_heads);
  const int64_t rest2 = rest / L.kv.n_kv_heads;
  uint16_t* base = static_cast<uint16_t*>((rest2 & 1) ? L.kv.v : L.kv.k) + (rest2 >> 1) * L.kv.layer_stride +
                   h * L.kv.head_stride + vec * 8;
  for (int j0 = 0; j0 < a; j0 += COMMIT_BATCH) {
    uint4 x[COMMIT_BATCH];
#pragma unroll
    for (int e = 0; e < COMMIT_BATCH; ++e)
      if (j0 + e < a && src[j0 + e] != dst[j0 + e]) x[e] = *reinterpret_cast<const uint4*>(base + src[j0 + e]);
#pragma unroll
    for (int e = 0; e < COMMIT_BATCH; ++e)
      if (j0 + e < a && src[j0 + e] != dst[j0 + e]) *reinterpret_cast<uint4*>(base + dst[j0 + e]) = x[e];
  }
}

template <typename T, int D>
cudaError_t append(const AppendLaunch& L, cudaStream_t stream) {
  constexpr int PER_CTA = APPEND_THREADS / (D / 8);
  const int chunks = (L.n_q_heads + 2 * L.kv.n_kv_heads + PER_CTA - 1) / PER_CTA;
  const int64_t ctas = static_cast<int64_t>(L.B) * L.nodes.count * chunks;
  return launch_pdl(kv_append_kernel<T, D>, dim3(static_cast<unsigned>(ctas)), dim3(APPEND_THREADS), 0, stream, L,
                    chunks, log2_of(L.kv.page_size));
}

}  // namespace

cudaError_t launch_kv_append(const AppendLaunch& L, cudaStream_t stream) {
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? append<__nv_bfloat16, 128>(L, stream) : append<__nv_bfloat16, 64>(L, stream);
  return L.kv.head_dim == 128 ? append<__half, 128>(L, stream) : append<__half, 64>(L, stream);
}

cudaError_t launch_kv_commit(const CommitLaunch& L, cudaStream_t stream) {
  const int vecs = L.kv.head_dim / 8;
  const int64_t lanes = static_cast<int64_t>(L.kv.n_layers) * 2 * L.kv.n_kv_heads * vecs;
  const int64_t ctas = (lanes + COMMIT_THREADS - 1) / COMMIT_THREADS;
  return launch_pdl(kv_commit_kernel, dim3(static_cast<unsigned>(ctas), L.B), dim3(COMMIT_THREADS), 0, stream, L,
                    lanes, vecs, log2_of(L.kv.page_size));
}

}  // namespace st
