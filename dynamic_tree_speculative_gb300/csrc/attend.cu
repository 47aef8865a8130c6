// Attention of a tree's nodes over a paged key-value cache of 16 bits
// (spec_tree_attend): keys and values come into shared memory by tensor map, as
// the tiles that the products take.
namespace st {
namespace {
constexpr bool CODES = false;
}
}  // namespace st

#include <algorithm>

#include "st_attend_tile.cuh"

namespace st {
namespace {

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    attend_kernel(const __grid_constant__ Plan P, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ CUtensorMap mq) {
  using Y = Layout<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem[];  // nothing static, so it starts on a swizzle group
  uint8_t* k_ring = smem + Y::Q_BYTES;
  uint8_t* v_ring = k_ring + Y::KS * Y::KV_BYTES;
  Control& C = *reinterpret_cast<Control*>(v_ring + Y::VS * Y::KV_BYTES);
  const int warp = __shfl_sync(FULL, threadIdx.x / 32, 0), cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_SLOTS; ++i) {
      mbar_init(&C.k_full[i], 1);
      mbar_init(&C.k_empty[i], 1);
      mbar_init(&C.v_full[i], 1);
      mbar_init(&C.v_empty[i], 2);  // the products' commit and the side warp
      mbar_init(&C.v_clean[i], 1);
    }
    mbar_init(&C.q_full, 1);
    mbar_init(&C.q_empty, 1);
    mbar_init(&C.drain, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&C.s_full[h], 1);
      mbar_init(&C.w_full[h][0], 4);
      mbar_init(&C.w_full[h][1], 4);
      mbar_init(&C.o_full[h], 1);
    }
    C.abort = 0;
    fence_mbar_init();
  }
  if (warp == HELPERS) tmem_alloc(&C.tmem, COLUMNS);
  if (threadIdx.x == THREADS - 1) {
    prefetch_map(&mk);
    prefetch_map(&mv);
    prefetch_map(&mq);
  }
  grid_dependency_wait();
  grid_dependents_launch();
  if (!P.may_piece || !find_piece<Y::HALVES>(P, C, C.tiles, cta)) find_range<Y::HALVES>(P, C, warp, cta);
  if (threadIdx.x == 0 && P.may_piece) workspace_of(P).records[cta].parts = 0;
  if (cta == 0)
    for (int b = threadIdx.x; b < P.L.B; b += THREADS) {
      int len, cnt;
      if (const uint32_t bad = tree_of(P, b, len, cnt)) set_status(P.L.status, bad);
    }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();

  if (warp < HELPERS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    softmax_role<T, D, PAIR>(P, C, smem, cta, static_cast<int>(min64(gridDim.x, C.total)), warp / 4);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(HELPER_REGS));
    if (warp == HELPERS) {
      load_role<D, PAIR, true>(P, &mk, C, smem_u32(k_ring));
    } else if (warp == HELPERS + 1) {
      load_role<D, PAIR, false>(P, &mv, C, smem_u32(v_ring));
    } else if (warp == HELPERS + 2) {
      product_role<T, D, PAIR>(P, C, smem_u32(smem), smem_u32(k_ring), smem_u32(v_ring));
      // products in flight end before their memory is given back, also where it
      // is the softmax that has given up and no longer waits for them
      if (elect()) mma_commit(&C.drain);
      __syncwarp();
      mbar_wait(&C.drain, 0);
    } else {
      side_role<T, D, PAIR>(P, &mq, C, smem_u32(smem), v_ring);
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == HELPERS) {
    tmem_fence_after();
    tmem_free(C.tmem, COLUMNS);
  }
}

// -------------------------------------------------------------------- host ---

// One layer's keys or values, [page][head][token][element]: `box` tokens of
// one head and page.
bool pool_map(CUtensorMap* map, const spec_tree_kv_t& kv, void* base, int layer, int box) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(kv.page_size),
                              static_cast<cuuint64_t>(kv.n_kv_heads), static_cast<cuuint64_t>(kv.n_pages)};
  const int64_t strides[3] = {kv.token_stride, kv.head_stride, kv.page_stride};
  return tiled_map(map, type_of(kv.dtype), 2, static_cast<uint16_t*>(base) + layer * kv.layer_stride, dims, strides,
                   {PANEL, static_cast<cuuint32_t>(box), 1, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int D, bool PAIR>
cudaError_t attend(Plan& P, cudaStream_t stream) {
  using Y = Layout<D, PAIR>;
  constexpr int SMEM = Y::Q_BYTES + (Y::KS + Y::VS) * Y::KV_BYTES + static_cast<int>(sizeof(Control));
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static_assert(2 * (TILE + D) <= COLUMNS, "tensor memory");
  const int item_rows = Y::HALVES * P.half_rows;
  P.row_tiles = (P.rows + item_rows - 1) / item_rows;
  P.ws_rows = std::min(P.rows, item_rows);
  const int64_t items = static_cast<int64_t>(P.L.B) * P.row_tiles;
  P.may_piece = items * P.L.kv.n_kv_heads <= P.L.num_sms && items <= MAX_PIECE_ITEMS;
  CUtensorMap mk, mv, mq;
  if (!pool_map(&mk, P.L.kv, P.L.kv.k, P.L.layer, P.box) || !pool_map(&mv, P.L.kv, P.L.kv.v, P.L.layer, P.box) ||
      !query_map(&mq, P))
    return cudaErrorInvalidValue;
  cudaError_t err = prepare_kernel<attend_kernel<T, D, PAIR>>(SMEM, LAUNCH_REGS);
  if (err != cudaSuccess) return err;
  err = launch_pdl(attend_kernel<T, D, PAIR>, dim3(P.L.num_sms), dim3(THREADS), SMEM, stream, P, mk, mv, mq);
  if (err != cudaSuccess || P.join_inside || !P.may_piece) return err;
  return launch_pdl(attend_join_kernel<T, D>, dim3(P.L.num_sms, JOIN_SLICES), dim3(JOIN_THREADS), 0, stream, P);
}

template <typename T, int D>
cudaError_t attend_rows(Plan& P, cudaStream_t stream) {
  return P.rows > P.half_rows ? attend<T, D, false>(P, stream) : attend<T, D, true>(P, stream);
}

int workspace_rows(int64_t rows) { return static_cast<int>(min64(rows, 2 * TILE)); }

}  // namespace

size_t attend_workspace_bytes(int num_sms, int64_t rows, int head_dim) {
  // up to `rows` rows; those that attend4_few.cu takes may have MAX_SPREAD CTAs on an SM
  const int many = workspace_rows(rows), few = static_cast<int>(min64(rows, SPEC_TREE_KV4_FEW_ROWS));
  const Workspace w = workspace_of(nullptr, num_sms, 0, 0);
  const size_t parts = static_cast<size_t>(num_sms) * 2 * std::max(many, MAX_SPREAD * few);
  return reinterpret_cast<size_t>(w.out) + parts * (sizeof(float2) + head_dim * 4);
}

cudaError_t launch_attend(const AttendLaunch& L, cudaStream_t stream) {
  Plan P = plan_of(L);
  P.q_box = std::min(TILE / P.group, L.nodes.count);
  P.box = L.kv.page_size < TILE ? L.kv.page_size : TILE;
  P.join_inside = P.rows <= JOIN_INSIDE_ROWS;
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend_rows<__nv_bfloat16, 128>(P, stream) : attend_rows<__nv_bfloat16, 64>(P, stream);
  return L.kv.head_dim == 128 ? attend_rows<__half, 128>(P, stream) : attend_rows<__half, 64>(P, stream);
}

}  // namespace st
