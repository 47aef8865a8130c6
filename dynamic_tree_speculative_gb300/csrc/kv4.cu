// A key-value cache in 4 bits: moving the accepted path behind the committed
// tokens (spec_tree_kv4_commit) and reading entries back (spec_tree_kv4_read).
#include "st_kernels.h"
#include "st_kv.cuh"

namespace st {
namespace {

constexpr int COMMIT_THREADS = 128;
constexpr int COMMIT_BATCH = 8;  // path steps loaded before any is stored
constexpr int READ_THREADS = 128;

// One thread per 16 bytes of a slot's codes, or per head's four scales and
// zeros, in one layer; as in the cache of 16 bits it walks the path in ascending
// order, COMMIT_BATCH steps at a time, loading a batch before storing it: step j
// reads slot path[j] >= j, which only a step after j may write.  One path of one layer
// takes 2.6 us, 16 of 32 layers 3.3 (1.7 MB): three dependent loads and a launch.
template <typename W>
__device__ __forceinline__ void move_path(uint8_t* base, const int64_t* src, const int64_t* dst, int steps, int shift) {
  for (int j0 = 0; j0 < steps; j0 += COMMIT_BATCH) {
    W x[COMMIT_BATCH];
#pragma unroll
    for (int e = 0; e < COMMIT_BATCH; ++e)
      if (j0 + e < steps && src[j0 + e] != dst[j0 + e]) x[e] = *reinterpret_cast<const W*>(base + (src[j0 + e] * 2 >> shift));
#pragma unroll
    for (int e = 0; e < COMMIT_BATCH; ++e)
      if (j0 + e < steps && src[j0 + e] != dst[j0 + e]) *reinterpret_cast<W*>(base + (dst[j0 + e] * 2 >> shift)) = x[e];
  }
}

__global__ void __launch_bounds__(COMMIT_THREADS) kv4_commit_kernel(const CommitLaunch L, int64_t lanes, int vecs, int page_shift) {
  // offsets of the path's entries: codes (in codes), scales and zeros (in elements)
  __shared__ int64_t src[2][256], dst[2][256];
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
      const int64_t from = static_cast<int64_t>(len) + node, to = static_cast<int64_t>(len) + j + 1;
      src[0][j] = kv_slot_offset(L.kv, b, from, page_shift);
      dst[0][j] = kv_slot_offset(L.kv, b, to, page_shift);
      if (src[0][j] < 0 || dst[0][j] < 0) {
        src[0][j] = dst[0][j] = src[1][j] = dst[1][j] = -1;
        set_status(L.status, SPEC_TREE_S_PAGES);
      } else {
        src[1][j] = kv_scale_offset(L.kv, L.scales, b, from, page_shift);
        dst[1][j] = kv_scale_offset(L.kv, L.scales, b, to, page_shift);
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
  // units of a head: its key's vectors, its value's, its scales and zeros
  const int units = 2 * vecs + 1;
  const int unit = static_cast<int>(t % units);
  const int64_t rest = t / units;
  const int h = static_cast<int>(rest % L.kv.n_kv_heads);
  const int64_t layer = rest / L.kv.n_kv_heads;
  if (unit < 2 * vecs) {
    const int64_t at = layer * L.kv.layer_stride + h * L.kv.head_stride + unit % vecs * 32;
    move_path<uint4>(static_cast<uint8_t*>(unit < vecs ? L.kv.k : L.kv.v) + at / 2, src[0], dst[0], a, 2);
  } else {
    const int64_t at = layer * L.scales.layer_stride + h * L.scales.head_stride;
    move_path<uint2>(static_cast<uint8_t*>(L.scales.data) + at * 2, src[1], dst[1], a, 0);
  }
}

// One warp takes 256 / D vectors of keys, then of values, at a time: a lane four
// bytes (8 codes) of one, which it writes as 16.  3904 entries of 8 heads of 128 (20 MB):
// 6.5 us, against 3.0 at the memory's rate; lookups before the loads are the rest.
template <typename T, int D>
__global__ void __launch_bounds__(READ_THREADS) kv4_read_kernel(const ReadLaunch L, int64_t vectors, int page_shift) {
  constexpr int LANES = D / 8;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t x = (static_cast<int64_t>(blockIdx.x) * READ_THREADS + threadIdx.x) / LANES;
  if (x >= vectors) return;
  const int lane = threadIdx.x % LANES, heads = L.kv.n_kv_heads;
  const int64_t entry = x / heads;
  const int h = static_cast<int>(x - entry * heads), b = static_cast<int>(entry / L.count);
  const int i = static_cast<int>(entry - static_cast<int64_t>(b) * L.count);
  int64_t off = -1;
  const int64_t slot = static_cast<int64_t>(L.first ? L.first[b] : 0) + i;
  const bool there = !L.counts || i < L.counts[b];
  if (there) off = kv_slot_offset(L.kv, b, slot, page_shift);
  if (there && off < 0 && h == 0 && lane == 0) set_status(L.status, SPEC_TREE_S_PAGES);
  uint32_t codes[2] = {0, 0};
  float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (off >= 0) {
    const int64_t at = (L.layer * L.kv.layer_stride + off + h * L.kv.head_stride + lane * 8) / 2;
    codes[0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(L.kv.k) + at);
    codes[1] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(L.kv.v) + at);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const T*>(L.scales.data) + L.layer * L.scales.layer_stride +
                                                    kv_scale_offset(L.kv, L.scales, b, slot, page_shift) +
                                                    h * L.scales.head_stride);
    const float2 k = Pair<T>::unpack(w.x), v = Pair<T>::unpack(w.y);
    sc[0] = k.x, sc[1] = k.y, sc[2] = v.x, sc[3] = v.y;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const spec_tree_heads_t& to = e == 0 ? L.k : L.v;
    float y[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) y[d] = fmaf(static_cast<float>((codes[e] >> (4 * d)) & 15u), sc[2 * e], sc[2 * e + 1]);
    *reinterpret_cast<uint4*>(static_cast<T*>(to.data) + b * to.tree_stride + i * to.node_stride + h * to.head_stride + lane * 8) =
        pack8<T>(y);
  }
}

template <typename T, int D>
cudaError_t read(const ReadLaunch& L, cudaStream_t stream) {
  const int64_t vectors = static_cast<int64_t>(L.B) * L.count * L.kv.n_kv_heads;
  const int64_t ctas = (vectors * (D / 8) + READ_THREADS - 1) / READ_THREADS;
  return launch_pdl(kv4_read_kernel<T, D>, dim3(static_cast<unsigned>(ctas)), dim3(READ_THREADS), 0, stream, L, vectors,
                    log2_of(L.kv.page_size));
}

}  // namespace

cudaError_t launch_kv4_commit(const CommitLaunch& L, cudaStream_t stream) {
  const int vecs = L.kv.head_dim / 32;
  const int64_t lanes = static_cast<int64_t>(L.kv.n_layers) * L.kv.n_kv_heads * (2 * vecs + 1);
  const int64_t ctas = (lanes + COMMIT_THREADS - 1) / COMMIT_THREADS;
  return launch_pdl(kv4_commit_kernel, dim3(static_cast<unsigned>(ctas), L.B), dim3(COMMIT_THREADS), 0, stream, L, lanes,
                    vecs, log2_of(L.kv.page_size));
}

cudaError_t launch_kv4_read(const ReadLaunch& L, cudaStream_t stream) {
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? read<__nv_bfloat16, 128>(L, stream) : read<__nv_bfloat16, 64>(L, stream);
  return L.kv.head_dim == 128 ? read<__half, 128>(L, stream) : read<__half, 64>(L, stream);
}

}  // namespace st
