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
// instead of NEW for 64 sequences of up to 5000 tokens; the integer pipe bounds it.)
//
// So queries and weights are f16 too, whatever the model's type.  Queries carry a
// power of two that brings the call's largest element near f16's; weights times
// values' scales one for each row, which goes down as larger scales come: both
// keep at least f16's 11 bits down to 2^-29 of the largest.
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
  // A lane's copies of a chunk: the same place in the page (or the two halves' pages), moved on from tile to tile.
  Walk<1> ahead(S);
  bool more = ahead.next(P);
  int tile = more ? ahead.s.first : 0;
  const int c = lane % LANES, token0 = lane / LANES;  // its first token, the others 32 / LANES apart
  const int64_t token_bytes = kv.token_stride / 2, page_bytes = kv.page_stride / 2, scale_page = P.L.scales.page_stride * 2;
  const bool small_pages = kv.page_size < CHUNK;  // 8 tokens: a chunk has two
  const uint8_t* key_at;                          // of page 0, entry 0 of the segment's head
  const uint8_t* scale_at;
  const int64_t to_values = static_cast<const uint8_t*>(kv.v) - static_cast<const uint8_t*>(kv.k);
  const int32_t* table;
  auto enter = [&] {  // a new segment
    key_at = static_cast<const uint8_t*>(kv.k) + (P.L.layer * kv.layer_stride + ahead.s.head * kv.head_stride) / 2 + c * 16;
    scale_at = static_cast<const uint8_t*>(P.L.scales.data) +
               (P.L.layer * P.L.scales.layer_stride + ahead.s.head * P.L.scales.head_stride) * 2;
    table = kv.page_table + static_cast<int64_t>(ahead.s.b) * kv.table_stride;
  };
  enter();
  int page[2] = {-1, -1};  // of the chunk's first and last 8 tokens
  auto look_up = [&] {
    const int slot = tile * TILE + warp * CHUNK;
    page[0] = page[1] = -1;
    if (more && slot < ahead.s.end) page[0] = page[1] = table[slot >> P.page_shift];
    if (small_pages && more) page[1] = slot + 8 < ahead.s.end ? table[(slot + 8) >> P.page_shift] : -1;
  };
  look_up();
  const uint32_t to_lane = smem_u32(ring) + token0 * (D / 2) + c * 16;
  // values: tokens in the order in which the products' lanes read them, so that these meet in few banks
  uint32_t to_value[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int token = token0 + i * (32 / LANES), row = (token & 8) | ((token & 1) << 2) | ((token >> 1) & 3);
    const int turn = D == 128 ? ((row >> 1) & 1) << 1 : 0;
    to_value[i] = smem_u32(ring) + F::CODE_BYTES + row * (D / 2) + ((c ^ turn) * 16);
  }
  auto load = [&](int stage) {  // the next chunk, if there is one; counts as a group in any case
    if (more) {
      const int slot = tile * TILE + warp * CHUNK, left = ahead.s.end - slot;  // tokens of the chunk and behind it
      const uint32_t skip = stage * F::STAGE_BYTES;
      const int entry = slot & (kv.page_size - 1);
      const bool ok[2] = {page[0] >= 0 && page[0] < kv.n_pages, page[1] >= 0 && page[1] < kv.n_pages};
      if ((!ok[0] && left > 0) || (!ok[1] && left > 8)) set_status(P.L.status, SPEC_TREE_S_PAGES);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int token = token0 + i * (32 / LANES);
        const int h = STEPS == 2 ? i : token / 8;  // two steps: a half each
        const bool there = (h ? ok[1] : ok[0]) && token < left;
        const uint8_t* from = key_at + (there ? (h ? page[1] : page[0]) : 0) * page_bytes +
                              (small_pages ? token % 8 : entry + token) * token_bytes;
        copy16(to_lane + skip + i * (32 / LANES) * (D / 2), from, there);
        copy16(to_value[i] + skip, from + to_values, there);
      }
      if (lane < CHUNK / 2) {
        const int token = 2 * lane;
        const bool second = lane >= CHUNK / 4, there = (second ? ok[1] : ok[0]) && token < left;
        copy16(smem_u32(ring) + skip + 2 * F::CODE_BYTES + lane * 16,
               scale_at + (there ? (second ? page[1] : page[0]) : 0) * scale_page + (small_pages ? token % 8 : entry + token) * 8, there);
      }
      if (++tile >= ahead.s.last) {
        more = ahead.next(P);
        tile = ahead.s.first;
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
    float scale_q;       // what a score's codes are multiplied by beside their scale
    {
      uint4 raw[NT][KEY_WORDS];
      float largest = 0.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + g, i = node_of_row(P, row);
        const T* from = static_cast<const T*>(P.L.q.data) + s.b * P.L.q.tree_stride + i * P.L.q.node_stride +
                        (static_cast<int64_t>(s.head) * P.group + row - i * P.group) * P.L.q.head_stride + t * 8 * KEY_WORDS;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KEY_WORDS; ++w) {
          raw[nt][w] = row < P.rows ? *reinterpret_cast<const uint4*>(from + 8 * w) : make_uint4(0, 0, 0, 0);
          float e[8];
          unpack8<T>(raw[nt][w], e);
#pragma unroll
          for (int d = 0; d < 8; ++d) sum += e[d], largest = fmaxf(largest, fabsf(e[d]));
        }
        sum += __shfl_xor_sync(FULL, sum, 1);
        sum += __shfl_xor_sync(FULL, sum, 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum_q[nt][e] = __shfl_sync(FULL, sum, (2 * t + e) * 4) * scale2;
          node[nt][e] = node_of_row(P, nt * 8 + 2 * t + e);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) largest = fmaxf(largest, __shfl_xor_sync(FULL, largest, o));
      const int e = min(exponent_above(largest), 126);
      const float up = power2(14 - e), up16 = power2(10 - e);
      scale_q = scale2 * power2(e - 14) * 16777216.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int w = 0; w < KEY_WORDS; ++w) {
          float x[8];
          unpack8<T>(raw[nt][w], x);
#pragma unroll
          for (int d = 0; d < 4; ++d)
            q[nt][2 * w + d / 2][d % 2] = Pair<__half>::pack(x[d] * (d % 2 ? up16 : up), x[d + 4] * (d % 2 ? up16 : up));
        }
    }
    float acc[NT][MT][4];               // outputs of elements x rows
    float sum[NT][2], middle[NT][2];    // of this lane's tokens: weights, weights times zeros
    float sub[NT][2], fit[NT][2];       // weights' reference; the power of two that goes with the values' scales
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) sum[nt][e] = middle[nt][e] = 0.0f, sub[nt][e] = -INFINITY, fit[nt][e] = power2(107);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][m][e] = 0.0f;
    }

    auto chunk = [&](auto is_masked, const uint8_t* at, int slot) {
      constexpr bool MASKED = decltype(is_masked)::value;
      // scales and zeros of tokens g and g + 8
      float ks[2], kz[2], vs[2], vz[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 w = *reinterpret_cast<const uint2*>(at + 2 * F::CODE_BYTES + (g + 8 * h) * 8);
        const float2 a = Pair<T>::unpack(w.x), b = Pair<T>::unpack(w.y);
        ks[h] = a.x * scale_q, kz[h] = a.y, vs[h] = b.x, vz[h] = b.y;
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
          const uint32_t a8 = a[w] >> 8, b8 = b[w] >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(dot[nt][0], a[w] & LOW, b[w] & LOW, a[w] & NEXT, b[w] & NEXT, q[nt][2 * w][0], q[nt][2 * w][1]);
            mma16816(dot[nt][1], a8 & LOW, b8 & LOW, a8 & NEXT, b8 & NEXT, q[nt][2 * w + 1][0], q[nt][2 * w + 1][1]);
          }
        }
      }
      uint32_t p[NT][2];  // the weights times scales, rows in the lanes
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // x[2 h + e]: token g + 8 h, row 2 t + e
        float x[4];
        bool seen[4];
        auto score = [&](int h, int e, float less) {
          return fmaf(ks[h], dot[nt][0][2 * h + e] + dot[nt][1][2 * h + e], fmaf(kz[h], sum_q[nt][e], -less));
        };
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[2 * h + e] = score(h, e, sub[nt][e]);  // infinity where there is no reference yet
            if (MASKED) {
              const int off = slot + g + 8 * h - s.len;
              bool see = off < 0;
              if (!see) {
                if (parent)
                  see = off < SPEC_TREE_MAX_NODES && ((S.sees[min(node[nt][e], MAX_NODES_FEW - 1)][off / 32] >> (off % 32)) & 1);
                else
                  see = off <= P.L.nodes.begin + node[nt][e];
              }
              if (!see) x[2 * h + e] = -INFINITY;
              seen[2 * h + e] = see;
            }
          }
        if (__any_sync(FULL, max3(x[0], x[1], fmaxf(x[2], x[3])) > LAZY)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool fresh = sub[nt][e] == -INFINITY;
            if (fresh) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (!MASKED || seen[2 * h + e]) x[2 * h + e] = score(h, e, 0.0f);
            }
            float top = fmaxf(x[e], x[2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
            if (fresh ? top > -INFINITY : top > LAZY) {
              const float f = fresh ? 0.0f : ex2(-top);
              sub[nt][e] = fresh ? top : sub[nt][e] + top;
              x[e] -= top, x[2 + e] -= top;
              sum[nt][e] *= f, middle[nt][e] *= f;
#pragma unroll
              for (int m = 0; m < MT; ++m) acc[nt][m][e] *= f, acc[nt][m][2 + e] *= f;
            }
          }
        }
        float w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = ex2(x[2 * h + e]);
            // what is not seen may hold anything
            const bool skip = MASKED && !seen[2 * h + e];
            sum[nt][e] += y;
            if (!skip) middle[nt][e] = fmaf(y, vz[h], middle[nt][e]);
            w[2 * h + e] = skip ? 0.0f : y * fit[nt][e] * vs[h];
          }
        if (__any_sync(FULL, max3(w[0], w[1], fmaxf(w[2], w[3])) > 32768.0f)) {
          // larger scales than before: at most 2^7 after this, weights at most 2^8
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (!MASKED || seen[2 * h + e]) top = fmaxf(top, vs[h]);
#pragma unroll
            for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
            const float next = fminf(fit[nt][e], power2(7 - exponent_above(top)));
            const float f = next / fit[nt][e];
            fit[nt][e] = next;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[2 * h + e] = MASKED && !seen[2 * h + e] ? 0.0f : ex2(x[2 * h + e]) * next * vs[h];
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[nt][m][e] *= f, acc[nt][m][2 + e] *= f;
          }
        }
        p[nt][0] = transposed(Pair<__half>::pack(w[0], w[1]));
        p[nt][1] = transposed(Pair<__half>::pack(w[2], w[3]));
      }
      // values: lane (g, t) has elements D / 8 g on of tokens 2 t, 2 t + 1, 2 t + 8 and 2 t + 9
      uint32_t v[4][VALUE_WORDS];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = (x & 2) * 4 + (x & 1) * 4 + t;
        const int turn = D == 128 ? ((row >> 1) & 1) << 1 : 0;
        lds<VALUE_WORDS>(v[x], at + F::CODE_BYTES + row * (D / 2) + (D == 128 ? (((g >> 1) ^ turn) * 16 + (g & 1) * 8) : g * 4));
      }
      uint32_t a[MT][4];  // two rows of each product, two pairs of tokens
#pragma unroll
      for (int w = 0; w < VALUE_WORDS; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __byte_perm(v[2 * h][w], v[2 * h + 1][w], 0x5410), hi = __byte_perm(v[2 * h][w], v[2 * h + 1][w], 0x7632);
          // word w of two, elements 0 .. 7: row g + 8 w of products 0 .. 7; of one word, elements 0 .. 3 and 4 .. 7: rows g, g + 8
          const int r = 2 * h + w, r2 = VALUE_WORDS == 2 ? r : 2 * h + 1, up = VALUE_WORDS == 2 ? 4 : 0;
          a[0][r] = lo & LOW, a[1][r] = lo & NEXT, a[2][r] = (lo >> 8) & LOW, a[3][r] = (lo >> 8) & NEXT;
          a[up][r2] = hi & LOW, a[up + 1][r2] = hi & NEXT, a[up + 2][r2] = (hi >> 8) & LOW, a[up + 3][r2] = (hi >> 8) & NEXT;
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < MT; ++m) mma16816(acc[nt][m], a[m][0], a[m][1], a[m][2], a[m][3], p[nt][0], p[nt][1]);
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
