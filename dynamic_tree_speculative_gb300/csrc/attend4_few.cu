// Attention over a key-value cache in 4 bits for calls of few rows: up to 16
// (nodes times query heads per key head), plain decoding above all.
//
// With a token's key s n + z and value s' n' + z' (n, n' codes), the scores are
// s (q . n) + z sum(q) and the outputs sum (w s') n' + sum w z': the codes
// themselves are multiplied, and scales and zeros are applied to the few products
// that leave.  A code in the lowest four bits of a 16-bit word is the f16 number
// n 2^-24, in the next four 16 n 2^-24: two codes of two of the eight in a word
// take one logic operation, and a shift by 8 serves the other four.  The factor 16
// goes into the queries, and out of the outputs at the end.  (As bf16 numbers 16 + n,
// each pair shifted to its place: 8 operations instead of 5 for 8 codes, and 121 us
// instead of 95 for one token of 64 sequences of 4500 on average; the integer pipe
// bounded it.)
//
// So queries and weights are f16 too, whatever the model's type.  Queries carry a
// power of two for each row, which brings its largest element near f16's; weights times
// values' scales one too, which goes down as larger scales come: both
// keep at least f16's 11 bits down to 2^-28 of the largest.
//
// Products are mma.sync, tokens (of keys) or elements (of values) in the rows and
// the call's rows in the columns, so that 8 rows fill a product: the codes go
// from shared memory to registers and into the product.  tcgen05 wants them
// unpacked in shared memory first, where 16-bit numbers cost 4.8 times the cache's
// own bytes to write and read, and pays off with rows to share that
// (attend4.cu).
//
// A warp takes 32 tokens of every other tile of 128 into a ring of its own (cp.async,
// no barriers); at the end of a segment the CTA's 8 warps put their sums together,
// while the next segment's loads are under way.  Tiles are dealt as in the
// attention over a cache of 16 bits.
//
// One token of 64 sequences of up to 5000 tokens, 32 query heads over 8 of 128 (286 MB: 42.7
// us at the measured bandwidth): 72 us, 57 with the products left out and 62 with the
// loads left out: 614 instructions a warp for 32 tokens of a key head, the issue slots 47 %
// and the integer pipe 41 % busy.  Without the rings (loads to registers as they were
// wanted) 95.  Two tokens over 131071 64 us with heads outermost, 66 with tokens, whose
// runs are 64 bytes.  16 rows instead of 4 take 116 us; 20, by attend4.cu, 182.
#include <type_traits>

#include "st_attend.cuh"

namespace st {
namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int BLOCK = 16;             // tokens of a product: its rows
constexpr int CHUNK = 2 * BLOCK;      // tokens of a warp's step
constexpr int SIDES = CHUNK * WARPS / TILE;  // half the warps take the even tiles of a segment, half the odd ones
constexpr int MAX_NODES_FEW = SPEC_TREE_KV4_FEW_ROWS;

template <int D, int NT>  // NT: products side by side, of 8 rows each
struct Few {
  static constexpr int CTAS = NT == 1 ? MAX_SPREAD : 1;  // on an SM
  static constexpr int STAGES = NT == 1 ? 2 : 4;
  static constexpr int CODE_BYTES = CHUNK * D / 2;             // of keys, and of values
  static constexpr int STAGE_BYTES = 2 * CODE_BYTES + CHUNK * 8;  // and scales and zeros
  static constexpr int RING_BYTES = WARPS * STAGES * STAGE_BYTES;
};

struct FewPlan : Plan {
  uint64_t token_bytes, page_bytes, scale_page_bytes;
  int64_t to_values;  // bytes from a key's codes to its value's
};

// The tiles that a side's warps load, one after the other.
struct Loads {
  int b, head, tile, last, tiles, end;
  int64_t left;  // tiles of the segments behind this one

  __device__ __forceinline__ Loads(const Plan& P, const Deal<WARPS>& C, int side) {
    const Segment& s = C.start;
    left = C.count;
    b = s.b, head = s.head, tiles = s.tiles, end = s.end;
    if (left <= 0) {
      last = 0, tile = 0;
      return;
    }
    const int n = static_cast<int>(min64(left, s.tiles - s.first));
    left -= n;
    tile = s.first + side, last = s.first + n;
    settle(P, side);
  }
  // on to the next segment that has a tile of the side, if there is one
  __device__ __forceinline__ void settle(const Plan& P, int side) {
    while (tile >= last && left > 0) {
      if (++head == P.L.kv.n_kv_heads) {
        head = 0, ++b;
        int len, cnt;
        tree_of(P, b, len, cnt);
        item_tiles<1>(P, len, cnt, 0, end, tiles);
      }
      last = static_cast<int>(min64(left, tiles));
      left -= last;
      tile = side;
    }
  }
  __device__ __forceinline__ bool more() const { return tile < last; }
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

// f16 products with float32 sums, 16 x 8 += 16 x 16 times 16 x 8.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr uint32_t LOW = 0x000f000fu, NEXT = 0x00f000f0u;  // codes n 2^-24 and 16 n 2^-24

__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The least e with x <= 2^e, of 2^-100 or more.
__device__ __forceinline__ int exponent_above(float x) {
  return static_cast<int>((__float_as_uint(fmaxf(x, power2(-100))) + 0x007fffffu) >> 23) - 127;
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // an 8 x 8 matrix of 16-bit numbers over the warp
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes into shared memory.  The L2 is to fetch 64 bytes around them, not the 128 that
// it does by itself: with heads inside tokens, the rest is of another head.  Two tokens
// over 131071: 94 -> 66 us; with heads outermost 64 either way.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ void copy16_or_zeros(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
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
__global__ void __launch_bounds__(THREADS, Few<D, NT>::CTAS) attend4_few_kernel(const __grid_constant__ FewPlan P) {
  using F = Few<D, NT>;
  constexpr int LANES = D / 32;          // that load a token's codes
  constexpr int TOKENS = 32 / LANES;     // of one step of loads
  constexpr int STEPS = BLOCK / TOKENS;  // of a block
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
  const int side = warp / (WARPS / SIDES), place = warp % (WARPS / SIDES) * CHUNK;  // the warp's tokens in a tile
  Loads ahead(P, S, side);
  const int c = lane % LANES, token0 = lane / LANES;  // a lane's first token; the others are TOKENS apart
  const uint8_t* key_at;    // the lane's part of token0, page 0, of the segment's head
  const uint8_t* scale_at;  // the lane's part of the scales of block 0 or 1
  const int32_t* table;
  auto enter = [&] {  // a new segment
    key_at = static_cast<const uint8_t*>(kv.k) + (P.L.layer * kv.layer_stride + ahead.head * kv.head_stride) / 2 +
             token0 * P.token_bytes + c * 16;
    scale_at = static_cast<const uint8_t*>(P.L.scales.data) +
               (P.L.layer * P.L.scales.layer_stride + ahead.head * P.L.scales.head_stride) * 2 + lane % (BLOCK / 2) * 16;
    table = kv.page_table + static_cast<int64_t>(ahead.b) * kv.table_stride;
  };
  enter();
  uint32_t page[2] = {0, 0};  // of the chunk's two blocks
  auto look_up = [&] {
    const int slot = ahead.tile * TILE + place;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (ahead.more() && slot + u * BLOCK < ahead.end) page[u] = table[(slot + u * BLOCK) >> P.page_shift];
  };
  look_up();
  const uint32_t ring_at = smem_u32(ring), to_key = ring_at + token0 * (D / 2) + c * 16;
  // values: tokens in the order in which the products' lanes read them, so that these meet in few banks
  const int value_row = (token0 & 8) | ((token0 & 1) << 2) | ((token0 >> 1) & 3);
  const int value_turn = D == 128 ? ((value_row >> 1) & 1) << 1 : 0;
  const uint32_t to_value = ring_at + F::CODE_BYTES + value_row * (D / 2) + ((c ^ value_turn) * 16);
  auto load = [&](int stage) {  // the next chunk, if there is one; counts as a group in any case
    if (ahead.more()) {
      const int slot = ahead.tile * TILE + place, left = ahead.end - slot;  // tokens of the chunk and behind it
      const uint32_t skip = stage * F::STAGE_BYTES, mask = kv.page_size - 1;
      const uint32_t pages = kv.n_pages;
      if (__builtin_expect(left >= CHUNK && page[0] < pages && page[1] < pages && kv.page_size >= BLOCK, 1)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t entry = (slot + u * BLOCK) & mask;
          const uint8_t* from = key_at + page[u] * P.page_bytes + entry * P.token_bytes;
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            const uint32_t to = skip + (u * STEPS + i) * TOKENS * (D / 2);
            copy16(to_key + to, from);
            copy16(to_value + to, from + P.to_values);
            from += TOKENS * P.token_bytes;
          }
        }
        if (lane < CHUNK / 2) {
          const int u = lane / (BLOCK / 2);
          copy16(ring_at + skip + 2 * F::CODE_BYTES + lane * 16,
                 scale_at + (u ? page[1] : page[0]) * P.scale_page_bytes + ((slot + u * BLOCK) & mask) * 8);
        }
      } else {
        // the end of the item, pages that are not in the pool, pages of 8 tokens
        auto page_of = [&](int token, bool& there) {
          const uint32_t x = token < left ? table[(slot + token) >> P.page_shift] : pages;
          if (x >= pages && token < left) set_status(P.L.status, SPEC_TREE_S_PAGES);
          there = x < pages;
          return there ? x : 0u;
        };
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i) {
          bool there;
          const uint64_t from_page = page_of(token0 + i * TOKENS, there) * P.page_bytes;
          const uint32_t to = skip + i * TOKENS * (D / 2), entry = (slot + token0 + i * TOKENS) & mask;
          const uint8_t* from = key_at + from_page + (static_cast<int64_t>(entry) - token0) * P.token_bytes;
          copy16_or_zeros(to_key + to, from, there);
          copy16_or_zeros(to_value + to, from + P.to_values, there);
        }
        if (lane < CHUNK / 2) {
          bool there;
          const uint64_t from_page = page_of(2 * lane, there) * P.scale_page_bytes;
          const int64_t entry = (slot + 2 * lane) & mask;
          copy16_or_zeros(ring_at + skip + 2 * F::CODE_BYTES + lane * 16,
                          scale_at + from_page + entry * 8 - lane % (BLOCK / 2) * 16, there);
        }
      }
      ahead.tile += SIDES;
      if (!ahead.more()) {
        ahead.settle(P, side);
        enter();
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
    // queries: lane (g, t) has a quarter of row g's elements, in the codes' order; those that meet 16 n are divided by 16
    uint32_t q[NT][2 * KEY_WORDS][2];
    float sum_q[NT][2];  // of rows 2 t and 2 t + 1
    int node[NT][2];     // theirs, among those of the call
    float scale_q[NT][2];  // what their scores' codes are multiplied by beside their scale
    {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + g, i = node_of_row(P, row);
        const T* from = static_cast<const T*>(P.L.q.data) + s.b * P.L.q.tree_stride + i * P.L.q.node_stride +
                        (static_cast<int64_t>(s.head) * P.group + row - i * P.group) * P.L.q.head_stride + t * 8 * KEY_WORDS;
        uint4 raw[KEY_WORDS];
        float sum = 0.0f, largest = 0.0f;
#pragma unroll
        for (int w = 0; w < KEY_WORDS; ++w) {
          raw[w] = row < P.rows ? *reinterpret_cast<const uint4*>(from + 8 * w) : make_uint4(0, 0, 0, 0);
          float e[8];
          unpack8<T>(raw[w], e);
#pragma unroll
          for (int d = 0; d < 8; ++d) sum += e[d], largest = fmaxf(largest, fabsf(e[d]));
        }
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
          sum += __shfl_xor_sync(FULL, sum, o);
          largest = fmaxf(largest, __shfl_xor_sync(FULL, largest, o));
        }
        const int exponent = min(exponent_above(largest), 126);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum_q[nt][e] = __shfl_sync(FULL, sum, (2 * t + e) * 4) * scale2;
          scale_q[nt][e] = scale2 * power2(__shfl_sync(FULL, exponent, (2 * t + e) * 4) - 14) * 16777216.0f;
          node[nt][e] = node_of_row(P, nt * 8 + 2 * t + e);
        }
        const float up = power2(14 - exponent), up16 = power2(10 - exponent);
#pragma unroll
        for (int w = 0; w < KEY_WORDS; ++w) {
          float x[8];
          unpack8<T>(raw[w], x);
#pragma unroll
          for (int d = 0; d < 4; ++d)
            q[nt][2 * w + d / 2][d % 2] = Pair<__half>::pack(x[d] * (d % 2 ? up16 : up), x[d + 4] * (d % 2 ? up16 : up));
        }
      }
    }
    float acc[NT][MT][4];               // outputs of elements x rows
    float sum[NT][2], middle[NT][2];    // of this lane's tokens: weights, weights times zeros
    float sub[NT][2], fit[NT][2];       // weights' reference; the power of two that goes with the values' scales
    float most[NT];                     // what a scale may be without a change of these
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      most[nt] = 128.0f / power2(107);
#pragma unroll
      for (int e = 0; e < 2; ++e) sum[nt][e] = middle[nt][e] = 0.0f, sub[nt][e] = -INFINITY, fit[nt][e] = power2(107);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][m][e] = 0.0f;
    }

    auto chunk = [&](auto is_masked, const uint8_t* at, int slot) {
      constexpr bool MASKED = decltype(is_masked)::value;
      // scales and zeros of tokens g and g + 8 of both blocks
      float ks[4], kz[4], vs[4], vz[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint2 w = *reinterpret_cast<const uint2*>(at + 2 * F::CODE_BYTES + (g + 8 * h) * 8);
        const float2 a = Pair<T>::unpack(w.x), b = Pair<T>::unpack(w.y);
        ks[h] = a.x, kz[h] = a.y, vs[h] = b.x, vz[h] = b.y;
      }
      float dot[NT][2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t a[KEY_WORDS], b[KEY_WORDS];
        lds<KEY_WORDS>(a, at + (u * BLOCK + g) * (D / 2) + t * (4 * KEY_WORDS));
        lds<KEY_WORDS>(b, at + (u * BLOCK + g + 8) * (D / 2) + t * (4 * KEY_WORDS));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) dot[nt][u][e] = 0.0f;
#pragma unroll
        for (int w = 0; w < KEY_WORDS; ++w) {
          const uint32_t a8 = a[w] >> 8, b8 = b[w] >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(dot[nt][u], a[w] & LOW, b[w] & LOW, a[w] & NEXT, b[w] & NEXT, q[nt][2 * w][0], q[nt][2 * w][1]);
            mma16816(dot[nt][u], a8 & LOW, b8 & LOW, a8 & NEXT, b8 & NEXT, q[nt][2 * w + 1][0], q[nt][2 * w + 1][1]);
          }
        }
      }
      uint32_t p[NT][4];  // the weights times scales, rows in the lanes
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // x[h][e]: token g + 8 h, row 2 t + e
        float x[4][2];
        bool seen[4][2];
        auto score = [&](int h, int e, float less) {
          return fmaf(ks[h] * scale_q[nt][e], dot[nt][h / 2][h % 2 * 2 + e], fmaf(kz[h], sum_q[nt][e], -less));
        };
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[h][e] = score(h, e, sub[nt][e]);  // infinity where there is no reference yet
            if (MASKED) {
              const int off = slot + g + 8 * h - s.len;
              bool see = off < 0;
              if (!see) {
                if (parent)
                  see = off < SPEC_TREE_MAX_NODES && ((S.sees[min(node[nt][e], MAX_NODES_FEW - 1)][off / 32] >> (off % 32)) & 1);
                else
                  see = off <= P.L.nodes.begin + node[nt][e];
              }
              if (!see) x[h][e] = -INFINITY;
              seen[h][e] = see;
            }
          }
        const float top_x = max3(max3(x[0][0], x[0][1], x[1][0]), max3(x[1][1], x[2][0], x[2][1]), fmaxf(x[3][0], x[3][1]));
        float top_s = max3(vs[0], vs[1], fmaxf(vs[2], vs[3]));
        if (MASKED) {
          top_s = 0.0f;
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (seen[h][0] || seen[h][1]) top_s = fmaxf(top_s, vs[h]);
        }
        if (__any_sync(FULL, top_x > LAZY || top_s > most[nt])) {
          most[nt] = INFINITY;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool fresh = sub[nt][e] == -INFINITY;
            float top = -INFINITY, larger = 0.0f;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              if (MASKED && !seen[h][e]) continue;
              if (fresh) x[h][e] = score(h, e, 0.0f);
              top = fmaxf(top, x[h][e]);
              larger = fmaxf(larger, vs[h]);
            }
#pragma unroll
            for (int o = 4; o < 32; o *= 2) {
              top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
              larger = fmaxf(larger, __shfl_xor_sync(FULL, larger, o));
            }
            float f = 1.0f;
            if (fresh ? top > -INFINITY : top > LAZY) {
              f = fresh ? 0.0f : ex2(-top);
              sub[nt][e] = fresh ? top : sub[nt][e] + top;
#pragma unroll
              for (int h = 0; h < 4; ++h) x[h][e] -= top;
              sum[nt][e] *= f, middle[nt][e] *= f;
            }
            // values' scales go up to 2^7, so weights times scales up to 2^15
            if (larger * fit[nt][e] > 128.0f) {
              const float next = power2(7 - exponent_above(larger));
              f *= next / fit[nt][e];
              fit[nt][e] = next;
            }
            most[nt] = fminf(most[nt], 128.0f / fit[nt][e]);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[nt][m][e] *= f, acc[nt][m][2 + e] *= f;
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = ex2(x[h][e]);
            // what is not seen may hold anything
            const bool skip = MASKED && !seen[h][e];
            sum[nt][e] += y;
            if (!skip) middle[nt][e] = fmaf(y, vz[h], middle[nt][e]);
            w[e] = skip ? 0.0f : y * fit[nt][e] * vs[h];
          }
          p[nt][h] = transposed(Pair<__half>::pack(w[0], w[1]));
        }
      }
      // values: lane (g, t) has elements D / 8 g on of tokens 2 t, 2 t + 1, 2 t + 8 and 2 t + 9 of each block
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t v[4][VALUE_WORDS];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = (x & 2) * 4 + (x & 1) * 4 + t;
          const int turn = D == 128 ? ((row >> 1) & 1) << 1 : 0;
          lds<VALUE_WORDS>(v[x], at + F::CODE_BYTES + (u * BLOCK + row) * (D / 2) +
                                     (D == 128 ? (((g >> 1) ^ turn) * 16 + (g & 1) * 8) : g * 4));
        }
        // pairs of tokens: elements 0 to 3 and 4 to 7 of a word
        uint32_t lo[VALUE_WORDS][2], hi[VALUE_WORDS][2];
#pragma unroll
        for (int w = 0; w < VALUE_WORDS; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            lo[w][h] = __byte_perm(v[2 * h][w], v[2 * h + 1][w], 0x5410);
            hi[w][h] = __byte_perm(v[2 * h][w], v[2 * h + 1][w], 0x7632);
          }
        // rows g and g + 8 of four products: of two words the first and the second, of one its halves
        auto four = [&](int m, const uint32_t (&a)[2], const uint32_t (&b)[2]) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t p0 = p[nt][2 * u], p1 = p[nt][2 * u + 1];
            mma16816(acc[nt][m], a[0] & LOW, b[0] & LOW, a[1] & LOW, b[1] & LOW, p0, p1);
            mma16816(acc[nt][m + 1], a[0] & NEXT, b[0] & NEXT, a[1] & NEXT, b[1] & NEXT, p0, p1);
            mma16816(acc[nt][m + 2], (a[0] >> 8) & LOW, (b[0] >> 8) & LOW, (a[1] >> 8) & LOW, (b[1] >> 8) & LOW, p0, p1);
            mma16816(acc[nt][m + 3], (a[0] >> 8) & NEXT, (b[0] >> 8) & NEXT, (a[1] >> 8) & NEXT, (b[1] >> 8) & NEXT, p0, p1);
          }
        };
        if (VALUE_WORDS == 2) {
          four(0, lo[0], lo[VALUE_WORDS - 1]);
          four(MT - 4, hi[0], hi[VALUE_WORDS - 1]);
        } else {
          four(0, lo[0], hi[0]);
        }
      }
    };

    for (int j = s.first + side; j < s.last; j += SIDES) {
      copies_wait<F::STAGES - 2>();
      __syncwarp();
      load(stage == 0 ? F::STAGES - 1 : stage - 1);  // the warp is done with the stage before
      const uint8_t* at = ring + stage * F::STAGE_BYTES;
      const int slot = j * TILE + place;
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
        if (g == 0) S.ref[warp][nt * 8 + 2 * t + e] = sub[nt][e];
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
        const float f = sub[nt][e] == -INFINITY ? (isnan(sum[nt][e]) ? 1.0f : 0.0f) : ex2(sub[nt][e] - top);
        if (g == 0) {
          S.sum[warp][row] = sum[nt][e] * f;
          if (warp == 0) S.top[row] = top;
        }
        // products of even numbers are of n 2^-24, odd ones of 16 n 2^-24
        const float out = middle[nt][e] * f, low = f * (16777216.0f / fit[nt][e]), next = f * (1048576.0f / fit[nt][e]);
        float* to = S.out[warp][row] + g * (D / 8);
#pragma unroll
        for (int m = 0; m < MT; m += 4)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float4*>(to + r * MT + m) =
                make_float4(fmaf(acc[nt][m][2 * r + e], low, out), fmaf(acc[nt][m + 1][2 * r + e], next, out),
                            fmaf(acc[nt][m + 2][2 * r + e], low, out), fmaf(acc[nt][m + 3][2 * r + e], next, out));
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
cudaError_t attend(FewPlan& P, cudaStream_t stream) {
  using F = Few<D, NT>;
  constexpr int SMEM = F::RING_BYTES + static_cast<int>(sizeof(FewShared<D, NT>));
  static_assert(F::CTAS * (SMEM + 1024) <= 233472, "shared memory of an SM");
  P.slots = F::CTAS * P.L.num_sms;
  P.may_piece = static_cast<int64_t>(P.L.B) * P.L.kv.n_kv_heads <= P.slots && P.L.B <= MAX_PIECE_ITEMS;
  const cudaError_t err = prepare_kernel<attend4_few_kernel<T, D, NT>>(SMEM, 0);
  if (err != cudaSuccess) return err;
  return launch_pdl(attend4_few_kernel<T, D, NT>, dim3(P.slots), dim3(THREADS), SMEM, stream, P);
}

template <typename T, int D>
cudaError_t attend_rows(FewPlan& P, cudaStream_t stream) {
  return P.rows <= 8 ? attend<T, D, 1>(P, stream) : attend<T, D, 2>(P, stream);
}

}  // namespace

cudaError_t launch_kv4_attend_few(const AttendLaunch& L, cudaStream_t stream) {
  FewPlan P;
  static_cast<Plan&>(P) = plan_of(L);
  P.token_bytes = L.kv.token_stride / 2;
  P.page_bytes = L.kv.page_stride / 2;
  P.scale_page_bytes = L.scales.page_stride * 2;
  P.to_values = static_cast<const uint8_t*>(L.kv.v) - static_cast<const uint8_t*>(L.kv.k);
  P.row_tiles = 1;
  P.ws_rows = P.rows;
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend_rows<__nv_bfloat16, 128>(P, stream) : attend_rows<__nv_bfloat16, 64>(P, stream);
  return L.kv.head_dim == 128 ? attend_rows<__half, 128>(P, stream) : attend_rows<__half, 64>(P, stream);
}

}  // namespace st
