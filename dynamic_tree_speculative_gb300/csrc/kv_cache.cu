// The paged key-value cache's writes: appending a tree's nodes with the head
// norms and the rotation on the way (spec_tree_kv_append), and moving the
// accepted path behind the committed tokens (spec_tree_kv_commit).
#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int APPEND_THREADS = 64, APPEND_BATCH = 4;  // heads whose loads a lane has in flight
// A node's heads are spread over warps until an SM has this many; a warp pays a
// node's lookups and rotation row once, so few with more heads each are faster:
// 8, 16 and 32 take 6.2, 9.2 and 10.0 us for 8 trees of 61 nodes (inputs past
// the L2), 11.3, 13.2 and 18.3 for 32, 19.7, 19.7 and 22.1 for 64.
constexpr int APPEND_WARPS = 8;
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

// One or more warps per node.  A head vector belongs to D / 16 neighbouring
// lanes, two chunks of 8 elements (16 bytes) each: the two that turn with each
// other (elements j and j + rot_dim / 2), or two neighbours where pairs are
// neighbours or nothing turns.  So a warp takes 4 or 8 vectors a step, pairs
// meet in their lane, and a lane's place in the vector, with it its part of the
// rotation row and of the weights, is the same in every step.
//
// With u the vector before the norm, w the weights and r = 1 / rms(u), a turned
// element is r (u_j (w_j c) + u_p (w_p s)), p its partner, s with the sign of
// j's place in the pair: the products in brackets are made once per node.
//
// Everything is read and written once; what bounds it is the issue rate and the
// loads in flight.  At 64 trees of 61 nodes of 48 heads of 128, normalised (95 MB:
// 14 us at the measured bandwidth): 19.6 us with inputs past the L2, 16 with them
// in it.  One chunk per lane, the partner's got by shuffles, took 24.5 (21.2 in
// the L2); one vector per thread, with a node's loads and products made for
// each, 37.2 in the L2.
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const __grid_constant__ AppendLaunch L, int page_shift,
                                                                   int nodes, int spread) {
  constexpr int LANES = D / 16, PER_STEP = 32 / LANES;
  const int lane = threadIdx.x % LANES, sub = threadIdx.x % 32 / LANES;
  const int warp = blockIdx.x * (APPEND_THREADS / 32) + threadIdx.x / 32;
  const int node = warp / spread;
  if (node >= nodes) return;
  const int n_q = L.n_q_heads, n_kv = L.kv.n_kv_heads;
  const int b = node / L.nodes.count, i = node - b * L.nodes.count, n = L.nodes.begin + i;
  const int half = L.rot_dim / 16;  // lanes whose chunks turn
  // the first elements of the lane's chunks
  const int e0 = 8 * (!INTERLEAVED && lane < half ? lane : 2 * lane);
  const int e1 = e0 + 8 * (!INTERLEAVED && lane < half ? half : 1);
  const T* q = static_cast<const T*>(L.q.data) + b * L.q.tree_stride + i * L.q.node_stride;
  const T* k = static_cast<const T*>(L.k.data) + b * L.k.tree_stride + i * L.k.node_stride;
  const T* w = static_cast<const T*>(L.v.data) + b * L.v.tree_stride + i * L.v.node_stride;
  T* q_to = static_cast<T*>(L.q_out.data) + b * L.q_out.tree_stride + i * L.q_out.node_stride;
  grid_dependency_wait();
  grid_dependents_launch();

  // a node's steps, dealt to its warps: the query heads first, then the key and
  // value heads (as one row); no step holds both, so one set of weighted
  // products lives at a time
  const int step0 = warp - node * spread, q_steps = (n_q + PER_STEP - 1) / PER_STEP;
  const int kv_step0 = (step0 < q_steps ? (q_steps - step0 + spread - 1) / spread * spread : 0) + step0 - q_steps;
  uint4 raw[APPEND_BATCH][2];
  auto load = [&](int u, const T* from) {
    raw[u][0] = *reinterpret_cast<const uint4*>(from + e0);
    raw[u][1] = *reinterpret_cast<const uint4*>(from + e1);
  };
  auto store = [&](T* to, const uint4 (&x)[2]) {
    *reinterpret_cast<uint4*>(to + e0) = x[0];
    *reinterpret_cast<uint4*>(to + e1) = x[1];
  };
  auto fetch = [&](bool queries, int step) {
#pragma unroll
    for (int u = 0; u < APPEND_BATCH; ++u) {
      const int head = (step + u * spread) * PER_STEP + sub;
      raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
      if (queries) {
        if (head < n_q) load(u, q + head * L.q.head_stride);
      } else if (head < n_kv) {
        load(u, k + head * L.k.head_stride);
      } else if (head < 2 * n_kv) {
        load(u, w + (head - n_kv) * L.v.head_stride);
      }
    }
  };
  fetch(true, step0);
  const int len = L.kv.seq_len[b], cnt = node_count(L.nodes, b);
  const int depth = L.nodes.depth ? L.nodes.depth[static_cast<int64_t>(b) * L.nodes.stride + n] : n;
  if (len < 0 && threadIdx.x % 32 == 0) set_status(L.status, SPEC_TREE_S_NODES);
  if (n >= cnt || len < 0) {
    const uint4 zeros[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    for (int head = step0 * PER_STEP + sub; head < n_q; head += spread * PER_STEP)
      store(q_to + head * L.q_out.head_stride, zeros);
    return;
  }
  const int64_t off = kv_slot_offset(L.kv, b, static_cast<int64_t>(len) + n, page_shift);
  if (off < 0 && threadIdx.x % 32 == 0) set_status(L.status, SPEC_TREE_S_PAGES);

  // the lane's 8 pairs' part of the rotation row
  const int64_t pos = static_cast<int64_t>(len) + depth;
  const bool turned = L.rot_dim > 0 && depth >= 0 && pos < L.rope_rows, turns = turned && lane < half;
  if (L.rot_dim > 0 && !turned && threadIdx.x % 32 == 0) set_status(L.status, SPEC_TREE_S_NODES);
  float4 c[2], s[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c[e] = make_float4(1.0f, 1.0f, 1.0f, 1.0f), s[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!turns) continue;
    const float* row = L.rope + pos * L.rot_dim + lane * 8 + 4 * e;
    c[e] = *reinterpret_cast<const float4*>(row);
    s[e] = *reinterpret_cast<const float4*>(row + L.rot_dim / 2);
  }
  auto flip = [](F2 x) {  // the other element of a neighbouring pair
    float lo, hi;
    x.get(lo, hi);
    return F2(hi, lo);
  };
  F2 cw[2][4], sw[2][4];  // with the weights of the heads in hand
  auto weighted = [&](const void* weight) {
    F2 x[2][4];
    if (weight != nullptr) {
      unpack_pairs<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + e0), x[0]);
      unpack_pairs<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + e1), x[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][e] = x[1][e] = F2(1.0f, 1.0f);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (INTERLEAVED) {
        cw[e][0] = mul2(x[e][0], F2(c[e].x, c[e].x)), sw[e][0] = mul2(flip(x[e][0]), F2(-s[e].x, s[e].x));
        cw[e][1] = mul2(x[e][1], F2(c[e].y, c[e].y)), sw[e][1] = mul2(flip(x[e][1]), F2(-s[e].y, s[e].y));
        cw[e][2] = mul2(x[e][2], F2(c[e].z, c[e].z)), sw[e][2] = mul2(flip(x[e][2]), F2(-s[e].z, s[e].z));
        cw[e][3] = mul2(x[e][3], F2(c[e].w, c[e].w)), sw[e][3] = mul2(flip(x[e][3]), F2(-s[e].w, s[e].w));
      } else {
        const F2 c0(c[e].x, c[e].y), c1(c[e].z, c[e].w), s0(s[e].x, s[e].y), s1(s[e].z, s[e].w);
        const F2 m0(-s[e].x, -s[e].y), m1(-s[e].z, -s[e].w);
        cw[0][2 * e] = mul2(x[0][2 * e], c0), cw[0][2 * e + 1] = mul2(x[0][2 * e + 1], c1);
        cw[1][2 * e] = mul2(x[1][2 * e], c0), cw[1][2 * e + 1] = mul2(x[1][2 * e + 1], c1);
        sw[0][2 * e] = mul2(x[1][2 * e], m0), sw[0][2 * e + 1] = mul2(x[1][2 * e + 1], m1);
        sw[1][2 * e] = mul2(x[0][2 * e], s0), sw[1][2 * e + 1] = mul2(x[0][2 * e + 1], s1);
      }
    }
  };
  // the vector normalised (if there are weights) and turned, in place; the whole
  // warp takes part in the sum, whatever its lanes hold
  auto turn = [&](uint4 (&u)[2], bool norm) {
    F2 x[2][4];
    unpack_pairs<T>(u[0], x[0]);
    unpack_pairs<T>(u[1], x[1]);
    F2 r(1.0f, 1.0f);
    if (norm) {
      F2 sum = mul2(x[0][0], x[0][0]), more = mul2(x[1][0], x[1][0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) sum = fma2(x[0][e], x[0][e], sum), more = fma2(x[1][e], x[1][e], more);
      float lo, hi;
      add2(sum, more).get(lo, hi);
      lo += hi;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) lo += __shfl_xor_sync(FULL, lo, o);
      lo = rsqrtf(lo * (1.0f / D) + L.eps);
      r = F2(lo, lo);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      F2 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = mul2(x[h][e], cw[h][e]);
        // elsewhere an infinity times the zero of s would be a NaN
        if (turns) y[e] = fma2(INTERLEAVED ? flip(x[h][e]) : x[1 - h][e], sw[h][e], y[e]);
        y[e] = mul2(y[e], r);
      }
      u[h] = pack_pairs<T>(y);
    }
  };

  weighted(L.q_weight);
  for (int at = step0; at < q_steps; at += APPEND_BATCH * spread) {
    if (at != step0) fetch(true, at);
#pragma unroll
    for (int u = 0; u < APPEND_BATCH; ++u) {
      const int head = (at + u * spread) * PER_STEP + sub;
      turn(raw[u], L.q_weight != nullptr);
      if (head < n_q) store(q_to + head * L.q_out.head_stride, raw[u]);
    }
  }
  weighted(L.k_weight);
  T* k_to = static_cast<T*>(L.kv.k) + L.layer * L.kv.layer_stride + off;
  T* v_to = static_cast<T*>(L.kv.v) + L.layer * L.kv.layer_stride + off;
  for (int at = kv_step0; at * PER_STEP < 2 * n_kv; at += APPEND_BATCH * spread) {
    fetch(false, at);
#pragma unroll
    for (int u = 0; u < APPEND_BATCH; ++u) {
      const int head = (at + u * spread) * PER_STEP + sub;
      if ((at + u * spread) * PER_STEP < n_kv) {  // uniform over the warp
        const uint4 v0 = raw[u][0], v1 = raw[u][1];
        turn(raw[u], L.k_weight != nullptr);
        if (head >= n_kv) raw[u][0] = v0, raw[u][1] = v1;  // a value beside keys
      }
      if (off >= 0) {
        if (head < n_kv)
          store(k_to + head * L.kv.head_stride, raw[u]);
        else if (head < 2 * n_kv)
          store(v_to + (head - n_kv) * L.kv.head_stride, raw[u]);
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

template <typename T, int D, bool INTERLEAVED>
cudaError_t append_as(const AppendLaunch& L, cudaStream_t stream) {
  constexpr int PER_STEP = 512 / D;
  const int nodes = L.B * L.nodes.count;
  const int steps = (L.n_q_heads + PER_STEP - 1) / PER_STEP + (2 * L.kv.n_kv_heads + PER_STEP - 1) / PER_STEP;
  int spread = 1;  // warps per node
  while (spread < steps && static_cast<int64_t>(nodes) * spread < L.num_sms * APPEND_WARPS) spread *= 2;
  if (spread > steps) spread = steps;
  const int64_t ctas = (static_cast<int64_t>(nodes) * spread + APPEND_THREADS / 32 - 1) / (APPEND_THREADS / 32);
  return launch_pdl(kv_append_kernel<T, D, INTERLEAVED>, dim3(static_cast<unsigned>(ctas)), dim3(APPEND_THREADS), 0, stream, L,
                    log2_of(L.kv.page_size), nodes, spread);
}

template <typename T, int D>
cudaError_t append(const AppendLaunch& L, cudaStream_t stream) {
  return L.interleaved ? append_as<T, D, true>(L, stream) : append_as<T, D, false>(L, stream);
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
