// Attention of a tree's nodes over a key-value cache in 4 bits
// (spec_tree_kv4_attend), for calls of more rows than attend4_few.cu takes: six
// warps unpack codes into the tiles that the products take, and the rest is as over a
// cache of 16 bits.
//
// Trees of 61 nodes after 4500 tokens, 64 sequences, take 252 us and a chunk of 2048
// tokens after 52 takes 120; with the arithmetic of unpacking left out 215 and 104 remained.
// Unpacking is bound by the integer pipe (5 operations for
// 8 codes, and 2 of f16 for each pair) and by shared memory (each 16-bit number is
// written once and read by each half of the rows), which the softmax's loads share.
namespace st {
namespace {
constexpr bool CODES = true;
}
}  // namespace st

#include <algorithm>

#include "st_attend_tile.cuh"

namespace st {
namespace {

constexpr int UNIT = 16, UNITS = TILE / UNIT;  // tokens that a warp unpacks together
constexpr int UNPACKERS = 6;                   // warps; no more than a tile has units, so that each sees every tile
static_assert(UNPACKERS <= UNITS, "a warp that does not see a tile may miss two phases of its barriers");

template <int D>
struct Raw {
  static constexpr int CODE_BYTES = UNIT * D / 2;
  static constexpr int BYTES = 2 * CODE_BYTES;
};

// 16 bytes, or zeros; the L2 fetches no more than 64 around them, which may be another head's.
__device__ __forceinline__ void copy_to_shared(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void copy8_to_shared(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(there ? 8 : 0) : "memory");
}

// Eight codes as s n + z, f16, j and j + 4 in word j.  A code in the lowest four bits of
// 1024 is 1024 + n, in the next four 1024 + 16 n; n is exact, and s n + z rounded once.
__device__ __forceinline__ uint4 unpacked(uint32_t w, __half2 s, __half2 z) {
  const __half2 low = __float2half2_rn(-1024.0f), next = __float2half2_rn(-64.0f), sixteenth = __float2half2_rn(0.0625f);
  uint32_t y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v = j < 2 ? w : w >> 8;
    const __half2 two = Pair<__half>::pair((v & (j % 2 ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u);
    const __half2 x = __hfma2(j % 2 ? __hfma2(two, sixteenth, next) : __hadd2(two, low), s, z);
    y[j] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// One warp: the tiles' scales and zeros, LEAD tiles ahead of their powers of two, which
// bring the largest element of the tile's 128 tokens, of keys and of values, near f16's; which values
// are not finite, where some rows may not see them, and zeros in their place; queries and
// parents.
template <typename T, int D, bool PAIR>
__device__ __forceinline__ void scale_role(const Plan& P, const CUtensorMap* mq, Control& C, uint32_t q_smem) {
  // 2 and 4 tiles ahead trees take as long, but 32 rows of 64 sequences of up to 5000 tokens
  // 246 and 250 us instead of 182
  constexpr int LEAD = 1;
  constexpr int EACH = TILE / 32;  // tokens of a lane; pages have 8 or more
  static_assert(EACH == 4, "a word of notes for 8 lanes");
  // Tiles of a segment that come before its queries are waited for, which are free once the
  // segment before is done with: that needs nothing of the segment itself as long as
  // the slot of the last of their loads is one of the segment before.
  constexpr int FIRST = SCALE_SLOTS - LEAD - 1;
  static_assert(FIRST >= 1, "slots");
  const spec_tree_kv_t& kv = P.L.kv;
  const int lane = threadIdx.x % 32;
  uint32_t* status = P.L.status;

  Walk<Layout<D, PAIR>::HALVES> ahead(C), walk(C);
  bool more = ahead.next(P);
  int to_load = ahead.s.first, page = -1;
  uint32_t loads = 0;
  auto look_up = [&] {
    const int slot = to_load * TILE + lane * EACH;
    page = more && slot < ahead.s.end ? kv.page_table[static_cast<int64_t>(ahead.s.b) * kv.table_stride + (slot >> P.page_shift)] : -1;
  };
  auto load = [&] {
    if (!more) return true;
    if (!warp_wait(&C.scale_empty[loads % SCALE_SLOTS], ((loads / SCALE_SLOTS) & 1) ^ 1, C, status)) return false;
    const int slot = to_load * TILE + lane * EACH;
    const bool ok = page >= 0 && page < kv.n_pages;
    if (!ok && slot < ahead.s.end) set_status(status, SPEC_TREE_S_PAGES);
    const uint8_t* from = static_cast<const uint8_t*>(P.L.scales.data) +
                          (P.L.layer * P.L.scales.layer_stride + ahead.s.head * P.L.scales.head_stride +
                           (ok ? page : 0) * P.L.scales.page_stride) * 2 + (slot & (kv.page_size - 1)) * 8;
    const uint32_t to = smem_u32(&C.scales[loads % SCALE_SLOTS][lane * EACH]);
#pragma unroll
    for (int x = 0; x < EACH; ++x) copy8_to_shared(to + x * 8, from + x * 8, ok && slot + x < ahead.s.end);
    ++loads;
    if (++to_load == ahead.s.last) {
      more = ahead.next(P);
      to_load = ahead.s.first;
    }
    look_up();
    return true;
  };
  look_up();
#pragma unroll 1
  for (int x = 0; x < LEAD; ++x) {
    load();
    commit_copies();
  }

  uint32_t segment = 0, n = 0, asked = 0;  // segments, tiles, segments whose queries have been asked for so far
  const Segment& s = walk.s;
  bool ok = true;
  for (; ok && walk.next(P); ++segment) {
    for (int j = s.first; ok; ++j, ++n) {
      if (asked == segment && (segment == 0 || j == min(s.first + FIRST, s.last))) {
        ok = ask_queries<D, PAIR>(P, mq, C, q_smem, s, segment);
        asked += ok;
      }
      if (!ok || j == s.last) break;
      ok = load();
      commit_copies();
      if (!ok) break;
      asm volatile("cp.async.wait_group %0;" ::"n"(LEAD) : "memory");
      uint2* mine = &C.scales[n % SCALE_SLOTS][lane * EACH];
      float key = 0.0f, value = 0.0f;
      uint32_t bad = 0;
      const bool masked = j >= s.clear / TILE;
#pragma unroll
      for (int x = 0; x < EACH; ++x) {
        const uint2 four = mine[x];
        const float2 k = Pair<T>::unpack(four.x);
        const float2 v = Pair<T>::unpack(four.y);
        const float most_k = fmaxf(fabsf(k.y), fabsf(fmaf(15.0f, k.x, k.y)));
        const float most_v = fmaxf(fabsf(v.y), fabsf(fmaf(15.0f, v.x, v.y)));
        if (isfinite(most_k)) key = fmaxf(key, most_k);
        if (isfinite(most_v)) value = fmaxf(value, most_v);
        if (masked && !(isfinite(v.x) && isfinite(v.y))) {
          bad |= 1u << x;
          mine[x].y = 0;
        }
      }
      if (masked) {
        const uint32_t word = __reduce_or_sync(0xffu << (lane / 8 * 8), bad << (lane % 8 * EACH));
        if (lane % 8 == 0) C.odd[segment % ODD_BUFFERS][(j - s.clear / TILE) * (TILE / 32) + lane / 8] = word;
      }
      // up to 2^14, which f16 holds with room for the roundings: what is 2^-28 as large keeps its 11 bits
      const int ek = -14 + power_above(__uint_as_float(__reduce_max_sync(FULL, __float_as_uint(key))));
      const int ev = -14 + power_above(__uint_as_float(__reduce_max_sync(FULL, __float_as_uint(value))));
      if (lane == 0)
        C.powers[n % POWER_SLOTS] = make_float4(P.scale2 * power2(ek), static_cast<float>(ev), power2(-ev), power2(-ek));
      warp_arrive(&C.scale_full[n % SCALE_SLOTS]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (asked > 0) mbar_wait(&C.q_full, (asked - 1) & 1);  // queries in flight land before the CTA ends
}

// One of UNPACKERS warps: every UNPACKERS-th unit, its codes into shared memory of the
// warp's own while the one before is unpacked into the tiles' rings.
template <typename T, int D, bool PAIR>
__device__ __forceinline__ void unpack_role(const Plan& P, Control& C, uint8_t* k_ring, uint8_t* v_ring, uint8_t* raw, int which) {
  using Y = Layout<D, PAIR>;
  using R = Raw<D>;
  constexpr int LANES = D / 32;       // for a token's codes
  constexpr int TOKENS = 32 / LANES;  // of one step of loads
  const spec_tree_kv_t& kv = P.L.kv;
  const int lane = threadIdx.x % 32, token = lane / LANES, c = lane % LANES;
  const uint64_t token_bytes = kv.token_stride / 2, page_bytes = kv.page_stride / 2;
  const uint32_t mask = kv.page_size - 1;
  raw += which * R::BYTES;
  uint32_t* status = P.L.status;

  // ---- loads
  Walk<Y::HALVES> walk(C);
  const Segment& s = walk.s;
  uint32_t before = 0;               // tiles of the segments before
  uint32_t ask = which;              // the unit to load next
  bool more = walk.next(P);
  int page[2] = {-1, -1};            // of its first and last 8 tokens
  const int64_t to_values = static_cast<const uint8_t*>(kv.v) - static_cast<const uint8_t*>(kv.k);
  const uint8_t* codes;              // of this lane's token, entry 0 of page 0 of the segment's head
  const int32_t* table;
  auto enter = [&] {
    codes = static_cast<const uint8_t*>(kv.k) + (P.L.layer * kv.layer_stride + s.head * kv.head_stride) / 2 + c * 16;
    table = kv.page_table + static_cast<int64_t>(s.b) * kv.table_stride;
  };
  auto slot_of = [&] { return (s.first + static_cast<int>(ask / UNITS - before)) * TILE + static_cast<int>(ask % UNITS) * UNIT; };
  auto look_up = [&] {  // on to the segment of `ask`, and its pages
    while (more && slot_of() >= s.last * TILE) {
      before += s.last - s.first;
      more = walk.next(P);
      enter();
    }
    page[0] = page[1] = -1;
    if (!more) return;
    const int slot = slot_of();
    if (slot < s.end) page[0] = page[1] = table[slot >> P.page_shift];
    if (kv.page_size < UNIT) page[1] = slot + 8 < s.end ? table[(slot + 8) >> P.page_shift] : -1;
  };
  enter();
  look_up();
  auto load = [&] {
    if (more) {
      const int slot = slot_of(), left = s.end - slot;
      const bool ok[2] = {page[0] >= 0 && page[0] < kv.n_pages, page[1] >= 0 && page[1] < kv.n_pages};
      const uint32_t to = smem_u32(raw);
#pragma unroll
      for (int i = 0; i < UNIT / TOKENS; ++i) {
        const int x = i * TOKENS + token, h = x / 8;
        const bool there = (h ? ok[1] : ok[0]) && x < left;
        const uint8_t* from = codes + static_cast<uint32_t>(there ? (h ? page[1] : page[0]) : 0) * page_bytes +
                              ((slot + x) & mask) * token_bytes;
        copy_to_shared(to + lane * 16 + i * 512, from, there);
        copy_to_shared(to + R::CODE_BYTES + lane * 16 + i * 512, from + to_values, there);
      }
      ask += UNPACKERS;
      look_up();
    }
  };
  load();

  // ---- tiles
  const uint32_t units = static_cast<uint32_t>(C.count) * UNITS;
  const int row_lane = lane / 2, half = lane % 2;
  for (uint32_t unit = which; unit < units; unit += UNPACKERS) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // a lane's token, and half of its codes: of 128 a panel's 64 elements, with neighbours beginning at different
    // halves, for the banks' sake
    uint4 key_words[D / 64], value_words[D / 64];
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      const int at = row_lane * (D / 2) + half * (D / 4) + (D == 128 ? (x ^ half) * 16 : 0);
      key_words[x] = *reinterpret_cast<const uint4*>(raw + at);
      value_words[x] = *reinterpret_cast<const uint4*>(raw + R::CODE_BYTES + at);
    }
    __syncwarp();
    load();  // the next unit, while this one is unpacked
    const uint32_t tile = unit / UNITS, in_tile = unit % UNITS;
    const int row = static_cast<int>(in_tile) * UNIT + row_lane;
    auto unpack = [&](uint8_t* to, const uint4 (&words)[D / 64], float2 pair, float down) {
      const __half2 scale = __float2half2_rn(pair.x * down), zero = __float2half2_rn(pair.y * down);
      to += row * 128 + (D == 128 ? half * PANEL_BYTES : 0);
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const uint32_t w[4] = {words[x].x, words[x].y, words[x].z, words[x].w};
        const int chunk = 4 * (D == 128 ? x ^ half : half);
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(to + (((chunk + i) ^ (row % 8)) << 4)) = unpacked(w[i], scale, zero);
      }
      fence_proxy_async_smem();
    };
    const uint32_t ks = tile % Y::KS, vs = tile % Y::VS;
    const uint32_t slot = tile % SCALE_SLOTS;
    if (!warp_wait(&C.scale_full[slot], (tile / SCALE_SLOTS) & 1, C, status)) break;
    const uint2 four = C.scales[slot][row];
    const float4 powers = C.powers[tile % POWER_SLOTS];
    if (!warp_wait(&C.k_empty[ks], ((tile / Y::KS) & 1) ^ 1, C, status)) break;
    unpack(k_ring + ks * Y::KV_BYTES, key_words, Pair<T>::unpack(four.x), powers.w);
    warp_arrive(&C.k_full[ks]);
    if (!warp_wait(&C.v_empty[vs], ((tile / Y::VS) & 1) ^ 1, C, status)) break;
    unpack(v_ring + vs * Y::KV_BYTES, value_words, Pair<T>::unpack(four.y), powers.z);
    warp_arrive(&C.v_full[vs]);
    warp_arrive(&C.scale_empty[slot]);  // so late, as the notes and the powers of the tiles behind it rest on it
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1) attend4_kernel(const __grid_constant__ Plan P, const __grid_constant__ CUtensorMap mq) {
  using Y = Layout<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem[];  // nothing static, so it starts on a swizzle group
  uint8_t* k_ring = smem + Y::Q_BYTES;
  uint8_t* v_ring = k_ring + Y::KS * Y::KV_BYTES;
  uint8_t* raw = v_ring + Y::VS * Y::KV_BYTES;
  Control& C = *reinterpret_cast<Control*>(raw + UNPACKERS * Raw<D>::BYTES);
  const int warp = __shfl_sync(FULL, threadIdx.x / 32, 0), cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_SLOTS; ++i) {
      mbar_init(&C.k_full[i], UNITS);
      mbar_init(&C.k_empty[i], 1);
      mbar_init(&C.v_full[i], UNITS);
      mbar_init(&C.v_empty[i], 1);
    }
    for (int i = 0; i < SCALE_SLOTS; ++i) {
      mbar_init(&C.scale_full[i], 1);
      mbar_init(&C.scale_empty[i], UNITS);
    }
    mbar_init(&C.q_full, 1);
    mbar_init(&C.q_empty, 1);
    mbar_init(&C.q_ready, HELPERS);
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
  if (threadIdx.x == THREADS - 1) prefetch_map(&mq);
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
      product_role<T, D, PAIR>(P, C, smem_u32(smem), smem_u32(k_ring), smem_u32(v_ring));
      // products in flight end before their memory is given back, also where it
      // is the softmax that has given up and no longer waits for them
      if (elect()) mma_commit(&C.drain);
      __syncwarp();
      mbar_wait(&C.drain, 0);
    } else if (warp == HELPERS + 1) {
      scale_role<T, D, PAIR>(P, &mq, C, smem_u32(smem));
    } else {
      unpack_role<T, D, PAIR>(P, C, k_ring, v_ring, raw, warp - HELPERS - 2);
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

template <typename T, int D, bool PAIR>
cudaError_t attend(Plan& P, cudaStream_t stream) {
  using Y = Layout<D, PAIR>;
  constexpr int SMEM = Y::Q_BYTES + (Y::KS + Y::VS) * Y::KV_BYTES + UNPACKERS * Raw<D>::BYTES + static_cast<int>(sizeof(Control));
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static_assert(2 * (TILE + D) <= COLUMNS, "tensor memory");
  static_assert(THREADS == (HELPERS + 2 + UNPACKERS) * 32, "roles");
  const int item_rows = Y::HALVES * P.half_rows;
  P.row_tiles = (P.rows + item_rows - 1) / item_rows;
  P.ws_rows = std::min(P.rows, item_rows);
  const int64_t items = static_cast<int64_t>(P.L.B) * P.row_tiles;
  P.may_piece = items * P.L.kv.n_kv_heads <= P.L.num_sms && items <= MAX_PIECE_ITEMS;
  CUtensorMap mq;
  if (!query_map(&mq, P)) return cudaErrorInvalidValue;
  cudaError_t err = prepare_kernel<attend4_kernel<T, D, PAIR>>(SMEM, LAUNCH_REGS);
  if (err != cudaSuccess) return err;
  err = launch_pdl(attend4_kernel<T, D, PAIR>, dim3(P.L.num_sms), dim3(THREADS), SMEM, stream, P, mq);
  if (err != cudaSuccess || !P.may_piece) return err;
  return launch_pdl(attend_join_kernel<T, D>, dim3(P.L.num_sms, JOIN_SLICES), dim3(JOIN_THREADS), 0, stream, P);
}

template <typename T, int D>
cudaError_t attend_rows(Plan& P, cudaStream_t stream) {
  return P.rows > P.half_rows ? attend<T, D, false>(P, stream) : attend<T, D, true>(P, stream);
}

}  // namespace

cudaError_t launch_kv4_attend(const AttendLaunch& L, cudaStream_t stream) {
  Plan P = plan_of(L);
  if (P.rows <= SPEC_TREE_KV4_FEW_ROWS) return launch_kv4_attend_few(L, stream);
  P.q_box = std::min(TILE / P.group, L.nodes.count);
  P.join_inside = false;
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend_rows<__nv_bfloat16, 128>(P, stream) : attend_rows<__nv_bfloat16, 64>(P, stream);
  return L.kv.head_dim == 128 ? attend_rows<__half, 128>(P, stream) : attend_rows<__half, 64>(P, stream);
}

}  // namespace st
