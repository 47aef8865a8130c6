// Attention over a key-value cache in 4 bits for calls of few rows: up to 16
// (nodes times query heads per key head), plain decoding above all.
//
// With a token's key s n + z and value s' n' + z' (n, n' codes), the scores are
// s (q . n) + z sum(q) and the outputs sum (w s') n' + sum w z': the codes
// themselves are multiplied, and scales and zeros are applied to the few products
// that leave.  A code's four bits, put into the mantissa of 16, are the 16-bit
// number 16 + n without any conversion: a shift and one three-input logic
// operation for two codes.  q . 16 goes back out with the zero; the values' 16,
// and 8 more so that what the weights' rounding multiplies is small, come out as
// 24 times the sum of the rounded weights, which a row of ones gives.
//
// Products are mma.sync, tokens (of keys) or elements (of values) in the rows and
// the call's rows in the columns, so that 8 rows fill a product: the codes go
// from shared memory to registers and into the product.  tcgen05 wants them
// unpacked in shared memory first, where 16-bit numbers cost 4.8 times the cache's
// own bytes to write and read, and pays off with rows to share that
// (attend4.cu).
//
// A warp takes 16 tokens of each tile of 128 into a ring of its own (cp.async, no
// barriers); at the end of a segment the CTA's 8 warps put their sums together,
// while the next segment's loads are under way.  Tiles are dealt as in the
// attention over a cache of 16 bits.
#include <type_traits>

#include "st_attend.cuh"

namespace st {
namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int CHUNK = TILE / WARPS;  // tokens of a warp's step: the rows of a product
constexpr int MAX_NODES_FEW = SPEC_TREE_KV4_FEW_ROWS;

template <int D, int NT>  // NT: products side by side, of 8 rows each
struct Few {
  static constexpr int CTAS = NT == 1 ? MAX_SPREAD : 1;  // on an SM
  static constexpr int STAGES = NT == 1 ? 4 : 8;
  static constexpr int CODE_BYTES = CHUNK * D / 2;             // of keys, and of values
  static constexpr int STAGE_BYTES = 2 * CODE_BYTES + CHUNK * 8;  // and scales and zeros
  static constexpr int RING_BYTES = WARPS * STAGES * STAGE_BYTES;
};

template <int D, int NT>
struct FewShared : Deal<WARPS> {
  alignas(16) float out[WARPS][8 * NT][D];
  float ref[WARPS][8 * NT], sum[WARPS][8 * NT], top[8 * NT];
  uint32_t sees[MAX_NODES_FEW][SPEC_TREE_MAX_NODES / 32];  // a node's ancestors and itself
  int16_t up[SPEC_TREE_MAX_NODES];
  int tiles[MAX_PIECE_ITEMS];
  int last;
};

// Codes J and J + 4 of eight as a pair of 16-bit numbers 16 + n.
template <typename T, int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  if (std::is_same<T, __half>::value) {
    w = J == 0 ? w << 6 : J == 1 ? w << 2 : J == 2 ? w >> 2 : w >> 6;
    return (w & 0x03c003c0u) | 0x4c004c00u;
  }
  w = J == 0 ? w << 3 : J == 1 ? w >> 1 : J == 2 ? w >> 5 : w >> 9;
  return (w & 0x00780078u) | 0x41804180u;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // an 8 x 8 matrix of 16-bit numbers over the warp
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes into shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups are there
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], const uint8_t* at) {
  if (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    w[0] = x.x, w[1] = x.y, w[N / 2] = x.z, w[N - 1] = x.w;
  } else if (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    w[0] = x.x, w[N - 1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(THREADS, Few<D, NT>::CTAS) attend4_few_kernel(const __grid_constant__ Plan P) {
  using F = Few<D, NT>;
  constexpr int LANES = D / 32;          // that load a token's codes
  constexpr int STEPS = D / 64;          // loads of a chunk
  constexpr int KEY_WORDS = D / 32;      // of a token, per lane
  constexpr int VALUE_WORDS = D / 64;
  constexpr int MT = D / 16;             // products of the outputs
  extern __shared__ __align__(1024) uint8_t smem[];
  FewShared<D, NT>& S = *reinterpret_cast<FewShared<D, NT>*>(smem + F::RING_BYTES);
  const int warp = __shfl_sync(FULL, threadIdx.x / 32, 0), lane = threadIdx.x % 32, cta = blockIdx.x;
  const int g = lane / 4, t = lane % 4;  // row and column pair of a product's lane
  uint8_t* ring = smem + warp * F::STAGES * F::STAGE_BYTES;
  const spec_tree_kv_t& kv = P.L.kv;

  grid_dependency_wait();
  grid_dependents_launch();
  if (!P.may_piece || !find_piece<1>(P, S, S.tiles, cta)) find_range<1>(P, S, warp, cta);
  if (cta == 0)
    for (int b = threadIdx.x; b < P.L.B; b += THREADS) {
      int len, cnt;
      if (const uint32_t bad = tree_of(P, b, len, cnt)) set_status(P.L.status, bad);
    }
  __syncthreads();

  // ------------------------------------------------------------------- loads ---
  Walk<1> ahead(S);
  bool more = ahead.next(P);
  int tile = more ? ahead.s.first : 0;
  int page[2] = {-1, -1};  // of the chunk's first and last 8 tokens
  auto look_up = [&] {
    page[0] = page[1] = -1;
    if (!more) return;
    const int slot = tile * TILE + warp * CHUNK;
    const int32_t* table = kv.page_table + static_cast<int64_t>(ahead.s.b) * kv.table_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (slot + 8 * h < ahead.s.end) page[h] = table[(slot + 8 * h) >> P.page_shift];
  };
  look_up();
  auto load = [&](int stage) {  // the next chunk, if there is one; counts as a group in any case
    if (more) {
      const int slot = tile * TILE + warp * CHUNK, end = ahead.s.end;
      const uint32_t to = smem_u32(ring + stage * F::STAGE_BYTES);
      bool there[2];
      int64_t base[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        there[h] = page[h] >= 0 && page[h] < kv.n_pages;
        if (!there[h] && slot + 8 * h < end) set_status(P.L.status, SPEC_TREE_S_PAGES);
        base[h] = there[h] ? page[h] : 0;
      }
      const int in_page = slot & (kv.page_size - 1), c = lane % LANES;
      const int64_t head = P.L.layer * kv.layer_stride + ahead.s.head * kv.head_stride;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int token = i * (32 / LANES) + lane / LANES;
        const bool second = token >= 8;
        const bool ok = (second ? there[1] : there[0]) && slot + token < end;
        // entry of the token in its page: pages of 8 tokens begin anew with the second half
        const int entry = (in_page + token) & (kv.page_size - 1);
        const int64_t at = head + (second ? base[1] : base[0]) * kv.page_stride + entry * kv.token_stride + c * 32;
        const uint32_t place = token * (D / 2) + c * 16;
        copy16(to + place, static_cast<const uint8_t*>(kv.k) + at / 2, ok);
        // values: tokens in the order in which the products' lanes read them, so that these meet in few banks
        const int row = (token & 8) | ((token & 1) << 2) | ((token >> 1) & 3);
        const int turn = D == 128 ? ((row >> 1) & 1) << 1 : 0;
        copy16(to + F::CODE_BYTES + row * (D / 2) + ((c ^ turn) * 16), static_cast<const uint8_t*>(kv.v) + at / 2, ok);
      }
      if (lane < CHUNK / 2) {
        const bool second = lane >= CHUNK / 4;
        const int token = 2 * lane, entry = (in_page + token) & (kv.page_size - 1);
        const int64_t at = P.L.layer * P.L.scales.layer_stride + (second ? base[1] : base[0]) * P.L.scales.page_stride +
                           ahead.s.head * P.L.scales.head_stride + entry * 4;
        copy16(to + 2 * F::CODE_BYTES + lane * 16, static_cast<const T*>(P.L.scales.data) + at,
               (second ? there[1] : there[0]) && slot + token < end);
      }
      if (++tile >= ahead.s.last) {
        more = ahead.next(P);
        tile = ahead.s.first;
      }
      look_up();
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < F::STAGES - 1; ++i) load(i);

  // ---------------------------------------------------------------- products ---
  const float scale2 = P.negative ? -P.scale2 : P.scale2;
  const int ctas = static_cast<int>(min64(gridDim.x, S.total));
  Walk<1> walk(S);
  const Segment& s = walk.s;
  int stage = 0;
  while (walk.next(P)) {
    const int32_t* parent = P.L.nodes.parent ? P.L.nodes.parent + static_cast<int64_t>(s.b) * P.L.nodes.stride : nullptr;
    if (parent && s.last * TILE > s.clear) {
      for (int x = threadIdx.x; x < s.cnt; x += THREADS) {
        const int up = parent[x];
        if (up >= x) set_status(P.L.status, SPEC_TREE_S_NODES);
        S.up[x] = static_cast<int16_t>(up < x ? max(up, -1) : -1);
      }
      for (int x = threadIdx.x; x < MAX_NODES_FEW * (SPEC_TREE_MAX_NODES / 32); x += THREADS) S.sees[0][x] = 0;
      __syncthreads();
      if (threadIdx.x < P.L.nodes.count)
        for (int at = P.L.nodes.begin + threadIdx.x; at >= 0 && at < s.cnt; at = S.up[at])
          S.sees[threadIdx.x][at / 32] |= 1u << (at % 32);
      __syncthreads();
    }
    // queries: lane (g, t) has a quarter of row g's elements, in the codes' order
    uint32_t q[NT][2 * KEY_WORDS][2];
    float sum_q[NT][2];  // of rows 2 t and 2 t + 1
    int node[NT][2];     // theirs, among those of the call
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g, i = node_of_row(P, row);
      const T* from = static_cast<const T*>(P.L.q.data) + s.b * P.L.q.tree_stride + i * P.L.q.node_stride +
                      (static_cast<int64_t>(s.head) * P.group + row - i * P.group) * P.L.q.head_stride + t * 8 * KEY_WORDS;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < KEY_WORDS; ++w) {
        const uint4 x = row < P.rows ? *reinterpret_cast<const uint4*>(from + 8 * w) : make_uint4(0, 0, 0, 0);
        float e[8];
        unpack8<T>(x, e);
#pragma unroll
        for (int d = 0; d < 8; ++d) sum += e[d];
        q[nt][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);
        q[nt][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
        q[nt][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);
        q[nt][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
      }
      sum += __shfl_xor_sync(FULL, sum, 1);
      sum += __shfl_xor_sync(FULL, sum, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum_q[nt][e] = __shfl_sync(FULL, sum, (2 * t + e) * 4);
        node[nt][e] = node_of_row(P, nt * 8 + 2 * t + e);
      }
    }
    float acc[NT][MT][4], ones[NT][4];       // outputs of elements x rows, sums of the rounded weights
    float sum[NT][2], middle[NT][2];         // of this lane's tokens: weights, weights times values' middles
    float sub[NT][2], allowed[NT][2];        // weights' reference, and what a score may exceed it by
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) sum[nt][e] = middle[nt][e] = sub[nt][e] = 0.0f, allowed[nt][e] = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ones[nt][e] = 0.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[nt][m][e] = 0.0f;
      }
    }

    auto chunk = [&](auto is_masked, const uint8_t* at, int slot) {
      constexpr bool MASKED = decltype(is_masked)::value;
      // scales and zeros of tokens g and g + 8
      float ks[2], kz[2], vs[2], vm[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 w = *reinterpret_cast<const uint2*>(at + 2 * F::CODE_BYTES + (g + 8 * h) * 8);
        const float2 a = Pair<T>::unpack(w.x), b = Pair<T>::unpack(w.y);
        ks[h] = a.x * scale2;
        kz[h] = fmaf(-16.0f, ks[h], a.y * scale2);
        vs[h] = b.x;
        vm[h] = fmaf(8.0f, b.x, b.y);
      }
      float dot[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) dot[nt][0][e] = dot[nt][1][e] = 0.0f;
      {
        uint32_t a[KEY_WORDS], b[KEY_WORDS];
        lds<KEY_WORDS>(a, at + g * (D / 2) + t * (4 * KEY_WORDS));
        lds<KEY_WORDS>(b, at + (g + 8) * (D / 2) + t * (4 * KEY_WORDS));
#pragma unroll
        for (int w = 0; w < KEY_WORDS; ++w) {
          const uint32_t a0 = code_pair<T, 0>(a[w]), a1 = code_pair<T, 1>(a[w]), a2 = code_pair<T, 2>(a[w]), a3 = code_pair<T, 3>(a[w]);
          const uint32_t b0 = code_pair<T, 0>(b[w]), b1 = code_pair<T, 1>(b[w]), b2 = code_pair<T, 2>(b[w]), b3 = code_pair<T, 3>(b[w]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<T>(dot[nt][0], a0, b0, a1, b1, q[nt][2 * w][0], q[nt][2 * w][1]);
            mma16816<T>(dot[nt][1], a2, b2, a3, b3, q[nt][2 * w + 1][0], q[nt][2 * w + 1][1]);
          }
        }
      }
      uint32_t p[NT][2];  // the weights times scales, rows in the lanes
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // x[2 h + e]: token g + 8 h, row 2 t + e
        float x[4];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[2 * h + e] = fmaf(ks[h], dot[nt][0][2 * h + e] + dot[nt][1][2 * h + e], fmaf(kz[h], sum_q[nt][e], -sub[nt][e]));
            if (MASKED) {
              const int off = slot + g + 8 * h - s.len;
              bool seen = off < 0;
              if (!seen) {
                if (parent)
                  seen = off < SPEC_TREE_MAX_NODES && ((S.sees[min(node[nt][e], MAX_NODES_FEW - 1)][off / 32] >> (off % 32)) & 1);
                else
                  seen = off <= P.L.nodes.begin + node[nt][e];
              }
              if (!seen) x[2 * h + e] = -INFINITY;
            }
            grow |= x[2 * h + e] > allowed[nt][e];
          }
        if (__any_sync(FULL, grow)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(x[e], x[2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
            if (top > allowed[nt][e]) {
              const float f = allowed[nt][e] == -INFINITY ? 0.0f : ex2(-top);
              sub[nt][e] += top;
              allowed[nt][e] = LAZY;
              x[e] -= top, x[2 + e] -= top;
              sum[nt][e] *= f, middle[nt][e] *= f;
              ones[nt][e] *= f, ones[nt][2 + e] *= f;
#pragma unroll
              for (int m = 0; m < MT; ++m) acc[nt][m][e] *= f, acc[nt][m][2 + e] *= f;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = ex2(x[2 * h + e]);
            // what is not seen may hold anything
            const bool skip = MASKED && x[2 * h + e] == -INFINITY;
            sum[nt][e] += y;
            middle[nt][e] = skip ? middle[nt][e] : fmaf(y, vm[h], middle[nt][e]);
            w[e] = skip ? 0.0f : y * vs[h];
          }
          p[nt][h] = transposed(Pair<__nv_bfloat16>::pack(w[0], w[1]));
        }
      }
      // values: lane (g, t) has elements D / 8 g on of tokens 2 t, 2 t + 1, 2 t + 8 and 2 t + 9
      uint32_t v[4][VALUE_WORDS];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = (x & 2) * 4 + (x & 1) * 4 + t;
        const int turn = D == 128 ? ((row >> 1) & 1) << 1 : 0;
        lds<VALUE_WORDS>(v[x], at + F::CODE_BYTES + row * (D / 2) + (D == 128 ? (((g >> 1) ^ turn) * 16 + (g & 1) * 8) : g * 4));
      }
      using H = __nv_bfloat16;
      uint32_t a[MT][4];  // two rows of each product, two pairs of tokens
#pragma unroll
      for (int w = 0; w < VALUE_WORDS; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __byte_perm(v[2 * h][w], v[2 * h + 1][w], 0x5410), hi = __byte_perm(v[2 * h][w], v[2 * h + 1][w], 0x7632);
          // word w of two, elements 0 .. 7: row g + 8 w of products 0 .. 7; of one word, elements 0 .. 3 and 4 .. 7: rows g, g + 8
          const int r = 2 * h + w, r2 = VALUE_WORDS == 2 ? r : 2 * h + 1, up = VALUE_WORDS == 2 ? 4 : 0;
          a[0][r] = code_pair<H, 0>(lo), a[1][r] = code_pair<H, 1>(lo), a[2][r] = code_pair<H, 2>(lo), a[3][r] = code_pair<H, 3>(lo);
          a[up][r2] = code_pair<H, 0>(hi), a[up + 1][r2] = code_pair<H, 1>(hi);
          a[up + 2][r2] = code_pair<H, 2>(hi), a[up + 3][r2] = code_pair<H, 3>(hi);
        }
      constexpr uint32_t ONES = 0x3f803f80u;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int m = 0; m < MT; ++m) mma16816<H>(acc[nt][m], a[m][0], a[m][1], a[m][2], a[m][3], p[nt][0], p[nt][1]);
        mma16816<H>(ones[nt], ONES, ONES, ONES, ONES, p[nt][0], p[nt][1]);
      }
    };

    for (int j = s.first; j < s.last; ++j) {
      copies_wait<F::STAGES - 2>();
      __syncwarp();
      load(stage == 0 ? F::STAGES - 1 : stage - 1);  // the warp is done with the stage before
      const uint8_t* at = ring + stage * F::STAGE_BYTES;
      const int slot = j * TILE + warp * CHUNK;
      if (slot + CHUNK <= s.clear && slot + CHUNK <= s.end)
        chunk(std::false_type(), at, slot);
      else if (slot < s.end)
        chunk(std::true_type(), at, slot);
      stage = stage + 1 == F::STAGES ? 0 : stage + 1;
    }

    // ------------------------------------------------------- the warps' sums ---
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          sum[nt][e] += __shfl_xor_sync(FULL, sum[nt][e], o);
          middle[nt][e] += __shfl_xor_sync(FULL, middle[nt][e], o);
        }
        if (g == 0) S.ref[warp][nt * 8 + 2 * t + e] = allowed[nt][e] == -INFINITY ? -INFINITY : sub[nt][e];
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * t + e;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, S.ref[w][row]);
        const float f = allowed[nt][e] == -INFINITY ? (isnan(sum[nt][e]) ? 1.0f : 0.0f) : ex2(sub[nt][e] - top);
        if (g == 0) {
          S.sum[warp][row] = sum[nt][e] * f;
          if (warp == 0) S.top[row] = top;
        }
        const float out = middle[nt][e] - 24.0f * ones[nt][e];
        float* to = S.out[warp][row] + g * (D / 8);
#pragma unroll
        for (int m = 0; m < MT; m += 4) {
          *reinterpret_cast<float4*>(to + m) = make_float4((acc[nt][m][e] + out) * f, (acc[nt][m + 1][e] + out) * f,
                                                           (acc[nt][m + 2][e] + out) * f, (acc[nt][m + 3][e] + out) * f);
          *reinterpret_cast<float4*>(to + MT + m) = make_float4((acc[nt][m][2 + e] + out) * f, (acc[nt][m + 1][2 + e] + out) * f,
                                                                (acc[nt][m + 2][2 + e] + out) * f, (acc[nt][m + 3][2 + e] + out) * f);
        }
      }
    __syncthreads();
    const bool whole = s.first == 0 && s.last == s.tiles;
    const Workspace ws = workspace_of(P);
    const int64_t part = cta * 2 + (s.first == 0 ? 1 : 0);
    for (int x = threadIdx.x; x < P.rows * (D / 4); x += THREADS) {
      const int row = x / (D / 4), d = x % (D / 4);
      float total = 0.0f;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(S.out[w][row] + 4 * d);
        total += S.sum[w][row];
        y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
      }
      const int i = node_of_row(P, row);
      const bool live = P.L.nodes.begin + i < s.cnt;
      if (!whole) {
        if (!live) continue;
        if (d == 0) ws.sums[part * P.ws_rows + row] = make_float2(S.top[row], total);
        ws.out[(part * (D / 4) + d) * P.ws_rows + row] = y;
      } else {
        const bool some = live && total != 0.0f;
        const float inv = some ? 1.0f / total : 0.0f;
        T* out = static_cast<T*>(P.L.out.data) + s.b * P.L.out.tree_stride + i * P.L.out.node_stride +
                 (static_cast<int64_t>(s.head) * P.group + row - i * P.group) * P.L.out.head_stride;
        *reinterpret_cast<uint2*>(out + 4 * d) =
            some ? make_uint2(Pair<T>::pack(y.x * inv, y.y * inv), Pair<T>::pack(y.z * inv, y.w * inv)) : make_uint2(0, 0);
      }
    }
    if (whole) continue;
    // the last CTA to leave its part of the item puts all of them together
    int from = cta, parts = 1;
    if (S.pieces) {
      from = cta - S.piece;
      parts = S.pieces;
    } else {
      if (s.first > 0) from = range_of(S.total, s.begin, ctas);
      parts = (s.last == s.tiles ? cta : range_of(S.total, s.begin + s.tiles - 1, ctas)) - from + 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* arrived = ws.arrived + from * 8;
      __threadfence();
      const bool last = atomicAdd(arrived, 1) + 1 == static_cast<uint32_t>(parts);
      __threadfence();
      if (last) *arrived = 0;
      S.last = last;
    }
    __syncthreads();
    if (S.last) join_rows<T, D>(P, ws, JoinRecord{parts, s.b, 0, s.head}, s.cnt, from, 0, P.rows, threadIdx.x, THREADS);
  }
  copies_wait<0>();
}

template <typename T, int D, int NT>
cudaError_t attend(Plan& P, cudaStream_t stream) {
  using F = Few<D, NT>;
  constexpr int SMEM = F::RING_BYTES + static_cast<int>(sizeof(FewShared<D, NT>));
  static_assert(F::CTAS * (SMEM + 1024) <= 233472, "shared memory of an SM");
  P.slots = F::CTAS * P.L.num_sms;
  P.may_piece = static_cast<int64_t>(P.L.B) * P.L.kv.n_kv_heads <= P.slots && P.L.B <= MAX_PIECE_ITEMS;
  const cudaError_t err = prepare_smem<attend4_few_kernel<T, D, NT>>(SMEM);
  if (err != cudaSuccess) return err;
  return launch_pdl(attend4_few_kernel<T, D, NT>, dim3(P.slots), dim3(THREADS), SMEM, stream, P);
}

template <typename T, int D>
cudaError_t attend_rows(Plan& P, cudaStream_t stream) {
  return P.rows <= 8 ? attend<T, D, 1>(P, stream) : attend<T, D, 2>(P, stream);
}

}  // namespace

cudaError_t launch_kv4_attend_few(const AttendLaunch& L, cudaStream_t stream) {
  Plan P = plan_of(L);
  P.row_tiles = 1;
  P.ws_rows = P.rows;
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend_rows<__nv_bfloat16, 128>(P, stream) : attend_rows<__nv_bfloat16, 64>(P, stream);
  return L.kv.head_dim == 128 ? attend_rows<__half, 128>(P, stream) : attend_rows<__half, 64>(P, stream);
}

}  // namespace st
