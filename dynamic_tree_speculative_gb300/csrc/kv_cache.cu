// The paged key-value cache's writes: appending a tree's nodes with the head
// norms and the rotation on the way (spec_tree_kv_append), and moving the
// accepted path behind the committed tokens (spec_tree_kv_commit).
#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int APPEND_THREADS = 128, APPEND_BATCH = 4;  // vectors a lane has in flight
constexpr int APPEND_WARPS = 32;                       // per SM, that a node's heads are spread over warps to reach
constexpr int COMMIT_THREADS = 128;
constexpr int COMMIT_BATCH = 8;  // path steps loaded before any is stored

// 16 bytes as four pairs of floats.
template <typename T>
__device__ __forceinline__ void unpack_pairs(uint4 w, F2 (&x)[4]) {
  x[0] = F2(Pair<T>::unpack(w.x));
  x[1] = F2(Pair<T>::unpack(w.y));
  x[2] = F2(Pair<T>::unpack(w.z));
  x[3] = F2(Pair<T>::unpack(w.w));
}

template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const F2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    x[e].get(lo, hi);
    w[e] = Pair<T>::pack(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One or more warps per node.  A head vector belongs to D / 8 neighbouring
// lanes, 8 elements (16 bytes) each, so a warp takes 2 or 4 vectors a step; a
// lane's place in the vector, and with it its part of the rotation row and of
// the weights, is the same in every step.
//
// With u the vector before the norm, w the weights and r = 1 / rms(u), a turned
// element is r (u_j (w_j c) + u_p (w_p s)), p its partner, s with the sign of
// j's place in the pair: the products in brackets are made once per node, and a
// lane gets its partners' u by shuffling the raw 16 bytes.
//
// Everything is read and written once; what bounds it is the issue rate.  At
// 64 trees of 61 nodes of 48 heads of 128, normalised (95 MB: 14 us at the
// measured bandwidth): 21.2 us (22.9 with queries' and keys' products held side
// by side and chosen per vector).  One vector per thread, with a node's loads and
// products made for each, took 37.2 us; three per thread 34.3 (253 instructions
// a step of a warp, of which this leaves 139).
template <typename T, int D>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const __grid_constant__ AppendLaunch L, int page_shift,
                                                                   int nodes, int spread) {
  constexpr int LANES = D / 8, PER_STEP = 32 / LANES;
  const int lane = threadIdx.x % LANES, sub = threadIdx.x % 32 / LANES;
  const int warp = blockIdx.x * (APPEND_THREADS / 32) + threadIdx.x / 32;
  const int node = warp / spread;
  if (node >= nodes) return;
  const int n_q = L.n_q_heads, n_kv = L.kv.n_kv_heads;
  const int b = node / L.nodes.count, i = node - b * L.nodes.count, n = L.nodes.begin + i;
  // pairs are elements j and j + rot_dim / 2, `half` lanes apart, or neighbours
  const int half = L.rot_dim / 16;
  const bool in_rot = lane < 2 * half, first = lane < half;
  const int partner = !in_rot || L.interleaved ? lane : (first ? lane + half : lane - half);
  const T* q = static_cast<const T*>(L.q.data) + b * L.q.tree_stride + i * L.q.node_stride + lane * 8;
  const T* k = static_cast<const T*>(L.k.data) + b * L.k.tree_stride + i * L.k.node_stride + lane * 8;
  const T* w = static_cast<const T*>(L.v.data) + b * L.v.tree_stride + i * L.v.node_stride + lane * 8;
  T* q_to = static_cast<T*>(L.q_out.data) + b * L.q_out.tree_stride + i * L.q_out.node_stride + lane * 8;
  grid_dependency_wait();
  grid_dependents_launch();

  // a node's steps, dealt to its warps: the query heads first, then the key and
  // value heads (as one row); no step holds both, so one set of weighted
  // products lives at a time
  const int step0 = warp - node * spread, q_steps = (n_q + PER_STEP - 1) / PER_STEP;
  const int kv_step0 = (step0 < q_steps ? (q_steps - step0 + spread - 1) / spread * spread : 0) + step0 - q_steps;
  uint4 raw[APPEND_BATCH];
  auto fetch = [&](bool queries, int step) {
#pragma unroll
    for (int u = 0; u < APPEND_BATCH; ++u) {
      const int head = (step + u * spread) * PER_STEP + sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (queries) {
        if (head < n_q) raw[u] = *reinterpret_cast<const uint4*>(q + head * L.q.head_stride);
      } else if (head < n_kv) {
        raw[u] = *reinterpret_cast<const uint4*>(k + head * L.k.head_stride);
      } else if (head < 2 * n_kv) {
        raw[u] = *reinterpret_cast<const uint4*>(w + (head - n_kv) * L.v.head_stride);
      }
    }
  };
  fetch(true, step0);
  const int len = L.kv.seq_len[b], cnt = node_count(L.nodes, b);
  const int depth = L.nodes.depth ? L.nodes.depth[static_cast<int64_t>(b) * L.nodes.stride + n] : n;
  if (len < 0 && threadIdx.x % 32 == 0) set_status(L.status, SPEC_TREE_S_NODES);
  if (n >= cnt || len < 0) {
    for (int step = step0; step * PER_STEP < n_q; step += spread)
      if (step * PER_STEP + sub < n_q)
        *reinterpret_cast<uint4*>(q_to + (step * PER_STEP + sub) * L.q_out.head_stride) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t off = kv_slot_offset(L.kv, b, static_cast<int64_t>(len) + n, page_shift);
  if (off < 0 && threadIdx.x % 32 == 0) set_status(L.status, SPEC_TREE_S_PAGES);

  // c and signed s of the lane's elements
  const int64_t pos = static_cast<int64_t>(len) + depth;
  const bool turned = L.rot_dim > 0 && depth >= 0 && pos < L.rope_rows;
  if (L.rot_dim > 0 && !turned && threadIdx.x % 32 == 0) set_status(L.status, SPEC_TREE_S_NODES);
  F2 c[4], s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = F2(1.0f, 1.0f), s[e] = F2(0.0f, 0.0f);
  const bool turns = turned && in_rot;
  if (turns) {
    const float* row = L.rope + pos * L.rot_dim;
    if (L.interleaved) {
      const float4 x = *reinterpret_cast<const float4*>(row + lane * 4);
      const float4 y = *reinterpret_cast<const float4*>(row + L.rot_dim / 2 + lane * 4);
      c[0] = F2(x.x, x.x), c[1] = F2(x.y, x.y), c[2] = F2(x.z, x.z), c[3] = F2(x.w, x.w);
      s[0] = F2(-y.x, y.x), s[1] = F2(-y.y, y.y), s[2] = F2(-y.z, y.z), s[3] = F2(-y.w, y.w);
    } else {
      const float* at = row + (first ? lane : lane - half) * 8;
      const float sign = first ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 x = *reinterpret_cast<const float4*>(at + 4 * e);
        const float4 y = *reinterpret_cast<const float4*>(at + L.rot_dim / 2 + 4 * e);
        c[2 * e] = F2(x.x, x.y), c[2 * e + 1] = F2(x.z, x.w);
        s[2 * e] = F2(sign * y.x, sign * y.y), s[2 * e + 1] = F2(sign * y.z, sign * y.w);
      }
    }
  }
  auto swapped = [&](uint4 x) {  // the other element of each neighbouring pair
    return make_uint4(__byte_perm(x.x, 0, 0x1032), __byte_perm(x.y, 0, 0x1032), __byte_perm(x.z, 0, 0x1032),
                      __byte_perm(x.w, 0, 0x1032));
  };
  F2 cw[4], sw[4];  // with the weights of the heads in hand
  auto weighted = [&](const void* weight) {
#pragma unroll
    for (int e = 0; e < 4; ++e) cw[e] = c[e], sw[e] = s[e];
    if (weight == nullptr) return;
    F2 x[4], y[4];
    unpack_pairs<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + lane * 8), x);
    const uint4 other = *reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + partner * 8);
    unpack_pairs<T>(L.interleaved ? swapped(other) : other, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) cw[e] = mul2(c[e], x[e]), sw[e] = mul2(s[e], y[e]);
  };
  // the vector normalised (if there are weights) and turned; the whole warp
  // takes part in the shuffles, whatever its lanes hold
  auto turn = [&](uint4 u, bool norm) {
    uint4 other = u;
    if (L.interleaved) {
      other = swapped(other);
    } else {
      other.x = __shfl_sync(FULL, other.x, partner, LANES);
      other.y = __shfl_sync(FULL, other.y, partner, LANES);
      other.z = __shfl_sync(FULL, other.z, partner, LANES);
      other.w = __shfl_sync(FULL, other.w, partner, LANES);
    }
    F2 x[4], y[4];
    unpack_pairs<T>(u, x);
    unpack_pairs<T>(other, y);
    F2 r(1.0f, 1.0f);
    if (norm) {
      F2 sum = mul2(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) sum = fma2(x[e], x[e], sum);
      float lo, hi;
      sum.get(lo, hi);
      lo += hi;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) lo += __shfl_xor_sync(FULL, lo, o);
      lo = rsqrtf(lo * (1.0f / D) + L.eps);
      r = F2(lo, lo);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = mul2(x[e], cw[e]);
      if (turns) x[e] = fma2(y[e], sw[e], x[e]);  // elsewhere an infinity times the zero of s would be a NaN
      x[e] = mul2(x[e], r);
    }
    return pack_pairs<T>(x);
  };

  weighted(L.q_weight);
  for (int at = step0; at < q_steps; at += APPEND_BATCH * spread) {
    if (at != step0) fetch(true, at);
#pragma unroll
    for (int u = 0; u < APPEND_BATCH; ++u) {
      const int head = (at + u * spread) * PER_STEP + sub;
      const uint4 y = turn(raw[u], L.q_weight != nullptr);
      if (head < n_q) *reinterpret_cast<uint4*>(q_to + head * L.q_out.head_stride) = y;
    }
  }
  weighted(L.k_weight);
  T* k_to = static_cast<T*>(L.kv.k) + L.layer * L.kv.layer_stride + off + lane * 8;
  T* v_to = static_cast<T*>(L.kv.v) + L.layer * L.kv.layer_stride + off + lane * 8;
  for (int at = kv_step0; at * PER_STEP < 2 * n_kv; at += APPEND_BATCH * spread) {
    fetch(false, at);
#pragma unroll
    for (int u = 0; u < APPEND_BATCH; ++u) {
      const int head = (at + u * spread) * PER_STEP + sub;
      uint4 y = raw[u];
      if ((at + u * spread) * PER_STEP < n_kv) y = turn(raw[u], L.k_weight != nullptr);  // uniform over the warp
      if (off >= 0) {
        if (head < n_kv)
          *reinterpret_cast<uint4*>(k_to + head * L.kv.head_stride) = y;
        else if (head < 2 * n_kv)
          *reinterpret_cast<uint4*>(v_to + (head - n_kv) * L.kv.head_stride) = raw[u];
      }
    }
  }
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
  constexpr int PER_STEP = 256 / D;
  const int nodes = L.B * L.nodes.count;
  const int steps = (L.n_q_heads + PER_STEP - 1) / PER_STEP + (2 * L.kv.n_kv_heads + PER_STEP - 1) / PER_STEP;
  int spread = 1;  // warps per node
  while (spread < steps && static_cast<int64_t>(nodes) * spread < L.num_sms * APPEND_WARPS) spread *= 2;
  if (spread > steps) spread = steps;
  const int64_t ctas = (static_cast<int64_t>(nodes) * spread + APPEND_THREADS / 32 - 1) / (APPEND_THREADS / 32);
  return launch_pdl(kv_append_kernel<T, D>, dim3(static_cast<unsigned>(ctas)), dim3(APPEND_THREADS), 0, stream, L,
                    log2_of(L.kv.page_size), nodes, spread);
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
