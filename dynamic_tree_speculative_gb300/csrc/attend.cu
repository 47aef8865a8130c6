// Attention of a tree's nodes over a paged key-value cache (spec_tree_attend).
//
// Rows.  The query heads that share a key head, over all nodes of the call,
// are the rows of one product: row r is node r / group, head r % group.  128
// rows make a half; calls of more than 128 rows work on two halves at a time,
// so that one half's softmax runs under the other half's products and keys
// and values are loaded once for both.
//
// Work.  An item is (tree, rows of 128 or 256, key head); its tokens are cut
// into tiles of 128.  All items' tiles, one after the other, are dealt to the
// CTAs (one per SM) in equal consecutive ranges, so a long cache is split over
// the card and a batch of ragged ones is balanced by the same rule.  An item
// whose tiles lie in one range is finished there; otherwise each range leaves
// its sums, their reference and its unnormalised output in the workspace, and
// attend_join_kernel puts the parts together in order.
//
// Tile.  S = Q K^T in tensor memory (128 lanes: one row per softmax thread);
// weights w = 2^(scale S - ref), rounded to the cache's type and stored over
// S; O += w V in tensor memory.  `ref` follows the row's maximum lazily: O is
// rescaled only when the maximum has grown by more than 2^8 since `ref` was
// set, so weights stay below 2^8 (f16: all weights carry another 2^7, so that
// small ones keep their bits) and the sums are the same up to rounding.
//
// Tokens a row does not see get S = -inf.  Their values enter the product
// with weight zero, so in tiles that not every row sees whole, infinities and
// NaN among the values are replaced by zero in shared memory first, and added
// at the end to the rows that do see them.
#include <cuda.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "st_kernels.h"
#include "st_kv.cuh"
#include "st_tensor.cuh"

namespace st {
namespace {

constexpr int TILE = 128;                       // tokens of a tile, rows of a half
constexpr int PANEL = 64;                       // elements of a 128-byte row
constexpr int PANEL_BYTES = TILE * 128;         // 128 rows of 64 elements
constexpr int MASKED_TILES = SPEC_TREE_MAX_NODES / TILE + 2;
constexpr float LAZY = 8.0f;                    // log2 of what a weight may exceed its reference by
constexpr int MAX_STAGES = 10;
constexpr int SPINS = 64;                       // polls of a wait before it suspends the thread

struct Plan {
  AttendLaunch L;
  int group, rows, row_tiles, page_shift, box, ws_rows;
  uint32_t group_inv;  // ceil(2^32 / group), 0 for a group of one
  float scale2;        // |scale| log2(e)
  bool negative;       // scale < 0: the products take -Q
};

// What a range has left in the workspace for the item it ends in, when others
// continue it: the join starts from there.
struct JoinRecord {
  int32_t pieces, b, row0, head;
};

struct Workspace {
  JoinRecord* records;  // [CTA]
  float2* sums;         // [CTA][2][ws_rows]: (reference, sum)
  float4* out;          // [CTA][2][D / 4][ws_rows]: neighbouring rows are neighbours in memory
};

__host__ __device__ inline Workspace workspace_of(void* ws, int num_sms, int ws_rows) {
  Workspace w;
  w.records = static_cast<JoinRecord*>(ws);
  w.sums = reinterpret_cast<float2*>(w.records + num_sms);
  w.out = reinterpret_cast<float4*>(w.sums + static_cast<size_t>(num_sms) * 2 * ws_rows);
  return w;
}

template <int D, int NH>
struct Layout {
  static constexpr int PANELS = D / PANEL;
  static constexpr int KV_BYTES = PANELS * PANEL_BYTES;
  static constexpr int Q_BYTES = NH * KV_BYTES;
  static constexpr int STAGES = (7 * 32768 - Q_BYTES) / KV_BYTES < MAX_STAGES ? (7 * 32768 - Q_BYTES) / KV_BYTES : MAX_STAGES;
  static constexpr int COLUMNS = NH * (TILE + D) > 256 ? 512 : 256;
  static constexpr int THREADS = (NH + 1) * TILE;
};

struct Control {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], clean[MAX_STAGES];
  uint64_t q_full, q_empty, s_full[2], w_full[2][2], o_full[2], drain;
  uint32_t tmem;
  int abort;
  int64_t scan[16];
  int64_t total;
  int b, rt, head, at;                       // where this CTA's range begins
  uint32_t odd[3][MASKED_TILES * (TILE / 32)];  // tokens with a value that is not finite, by segment modulo 3
  uint16_t parent[2][SPEC_TREE_MAX_NODES];      // by segment modulo 2
};

// A consecutive piece of an item's tiles: what one CTA does at a time.
struct Segment {
  int b, head, row0;     // row0: first row of the item
  int len, cnt;          // committed tokens, nodes that exist
  int first, last, tiles;  // tiles first .. last - 1 of `tiles`
  int end;               // tokens (slots) the item reads
  int clear;             // slots below this one are seen by every row of the item
};

// Committed tokens and nodes of tree b; none of either (and a status bit) for
// a length below zero or slots past the page table.
__device__ __forceinline__ uint32_t tree_of(const Plan& P, int b, int& len, int& cnt) {
  len = P.L.kv.seq_len[b];
  cnt = node_count(P.L.nodes, b);
  const uint32_t bad = len < 0 ? SPEC_TREE_S_NODES
                       : static_cast<int64_t>(len) + cnt > (static_cast<int64_t>(P.L.kv.max_pages) << P.page_shift)
                           ? SPEC_TREE_S_PAGES
                           : 0u;
  if (bad) len = 0, cnt = 0;
  return bad;
}

template <int NH>
__device__ __forceinline__ void item_tiles(const Plan& P, int len, int cnt, int rt, int& end, int& tiles) {
  const int last_row = min((rt + 1) * NH * TILE, P.rows) - 1;
  const int nodes = min(cnt, P.L.nodes.begin + last_row / P.group + 1);
  const int first = P.L.nodes.begin + rt * NH * TILE / P.group;
  end = first < cnt ? len + nodes : 0;  // rows of nodes that do not exist read nothing
  tiles = end > 0 ? (end + TILE - 1) / TILE : 1;
}

template <int NH>
__device__ __forceinline__ int64_t tree_tiles(const Plan& P, int b) {
  int len, cnt;
  tree_of(P, b, len, cnt);
  int64_t sum = 0;
  for (int rt = 0; rt < P.row_tiles; ++rt) {
    int end, tiles;
    item_tiles<NH>(P, len, cnt, rt, end, tiles);
    sum += tiles;
  }
  return sum * P.L.kv.n_kv_heads;
}

__device__ __forceinline__ int64_t range_start(int64_t total, int c, int ctas) { return total * c / ctas; }

// The segments of a CTA's range, one after the other; every role walks them
// for itself.
template <int NH>
struct Walk {
  int b, rt, head, at;
  int64_t left;
  int len, cnt;

  __device__ __forceinline__ void begin(const Plan& P, const Control& C, int64_t tiles) {
    left = tiles;
    if (left <= 0) return;
    b = C.b;
    rt = C.rt;
    head = C.head;
    at = C.at;
    tree_of(P, b, len, cnt);
  }

  __device__ __forceinline__ bool next(const Plan& P, Segment& s) {
    if (left <= 0) return false;
    s.b = b;
    s.head = head;
    s.row0 = rt * NH * TILE;
    s.len = len;
    s.cnt = cnt;
    item_tiles<NH>(P, len, cnt, rt, s.end, s.tiles);
    s.clear = P.L.nodes.parent ? len : len + min(cnt, P.L.nodes.begin + s.row0 / P.group + 1);
    s.first = at;
    const int64_t n = min64(left, s.tiles - at);
    s.last = at + static_cast<int>(n);
    left -= n;
    at = 0;
    if (s.last == s.tiles && ++head == P.L.kv.n_kv_heads) {
      head = 0;
      if (++rt == P.row_tiles) {
        rt = 0;
        if (left > 0) tree_of(P, ++b, len, cnt);
      }
    }
    return true;
  }
};

// Row `row0` + r of an item: node i0 + (rem + r) / group of the call, head
// (rem + r) % group.  rem + r < 2^15, so the product with the rounded-up
// inverse is exact.
struct Rows {
  int i0, rem;
  __device__ __forceinline__ Rows(const Plan& P, int row0) : i0(row0 / P.group), rem(row0 - row0 / P.group * P.group) {}
  __device__ __forceinline__ void get(const Plan& P, int r, int& i, int& g) const {
    const int x = rem + r;
    const int n = P.group_inv ? static_cast<int>(__umulhi(x, P.group_inv)) : x;
    i = i0 + n;
    g = x - n * P.group;
  }
};

// A wait that gives up when it, or another role of the CTA, has run out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Control& C, uint32_t* status) {
  const uint32_t addr = smem_u32(bar);
  uint32_t done;
  for (int spin = 0; spin < SPINS; ++spin) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
  }
  for (uint32_t it = 0; it < WAIT_LIMIT; ++it) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(addr), "r"(parity), "r"(WAIT_SUSPEND_NS)
        : "memory");
    if (done) return true;
    if (*reinterpret_cast<volatile int*>(&C.abort)) return false;
  }
  *reinterpret_cast<volatile int*>(&C.abort) = 1;
  set_status(status, SPEC_TREE_S_TIMEOUT);
  return false;
}

// The same for a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Control& C, uint32_t* status) {
  return __all_sync(FULL, wait(bar, parity, C, status));
}

// One arrival for a whole warp, after what all its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// bit j: the row's node sees slot `base` + j of the 128 slots of a tile
struct Seen {
  uint32_t w[TILE / 32];
};

__device__ __forceinline__ uint32_t below(int n) {  // the n lowest bits, n clamped to 0 .. 32
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

template <typename Parent>  // Parent(n): -1 for none
__device__ __forceinline__ Seen seen_of(const Plan& P, const Segment& s, int node, int base, Parent parent) {
  Seen v;
  const int off = base - s.len;  // node index of the tile's first slot
  const int prefix = P.L.nodes.parent ? -off : node + 1 - off;
#pragma unroll
  for (int i = 0; i < TILE / 32; ++i) v.w[i] = below(prefix - 32 * i);
  if (P.L.nodes.parent) {
    int at = node;
    while (at >= 0 && at >= off) {
      const int j = at - off;
#pragma unroll
      for (int i = 0; i < TILE / 32; ++i)
        if ((j >> 5) == i) v.w[i] |= 1u << (j & 31);
      at = parent(at);
    }
  }
  return v;
}

template <typename T>
__device__ __forceinline__ bool odd16(uint32_t h) {  // infinity or NaN in the low half
  constexpr uint32_t E = sizeof(T) == 2 && std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (h & E) == E;
}

// ------------------------------------------------------------------- roles ---

// One warp: tokens' keys and values from their pages into the ring, K and V
// of a tile one after the other.  Lane i copies the tile's i-th page (or its
// 128 tokens of a larger one); pages past the item's end are not read.
template <int D, int NH>
__device__ __forceinline__ void load_role(const Plan& P, const CUtensorMap* mk, const CUtensorMap* mv, Control& C,
                                          uint32_t ring, int64_t my_tiles) {
  using Y = Layout<D, NH>;
  const int lane = threadIdx.x % 32;
  const int boxes = TILE / P.box;
  Walk<NH> walk;
  walk.begin(P, C, my_tiles);
  Segment s;
  uint32_t n = 0;  // loads so far
  while (walk.next(P, s)) {
    const int32_t* table = P.L.kv.page_table + static_cast<int64_t>(s.b) * P.L.kv.table_stride;
    for (int t = s.first; t < s.last; ++t) {
      const int slot = t * TILE + lane * P.box;
      const bool mine = lane < boxes && slot < s.end;
      int page = P.L.kv.n_pages;  // outside the pool: the copy fills zeros
      if (mine) {
        const int idx = slot >> P.page_shift;
        const int got = idx < P.L.kv.max_pages ? table[idx] : -1;
        if (got >= 0 && got < P.L.kv.n_pages)
          page = got;
        else
          set_status(P.L.status, SPEC_TREE_S_PAGES);
      }
      const int off = slot & (P.L.kv.page_size - 1);
      const int used = s.end > 0 ? min(boxes, (s.end - t * TILE + P.box - 1) / P.box) : 0;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++n) {
        const int st = n % Y::STAGES;
        if (!warp_wait(&C.empty[st], ((n / Y::STAGES) & 1) ^ 1, C, P.L.status)) {
          // copies in flight land before the CTA ends
          for (uint32_t o = n > Y::STAGES ? n - Y::STAGES : 0; o < n; ++o)
            mbar_wait(&C.full[o % Y::STAGES], (o / Y::STAGES) & 1);
          return;
        }
        if (lane == 0) mbar_expect_tx(&C.full[st], used * P.box * 128 * Y::PANELS);
        __syncwarp();
        if (mine) {
#pragma unroll
          for (int p = 0; p < Y::PANELS; ++p)
            tile_g2s(ring + st * Y::KV_BYTES + p * PANEL_BYTES + lane * P.box * 128, kv ? mv : mk, p * PANEL, off,
                     s.head, page, &C.full[st]);
        }
      }
    }
  }
}

// One warp: the products.  The halves take turns, so that while one half's
// weights are made the other half's products run.  False: a wait gave up.
template <typename T, int D, int NH>
__device__ __forceinline__ bool product_role(const Plan& P, Control& C, uint32_t q_smem, uint32_t ring, int64_t my_tiles) {
  using Y = Layout<D, NH>;
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t ID_S = mma_descriptor(BF, TILE, false), ID_O = mma_descriptor(BF, D, true);
  constexpr int KV16 = Y::KV_BYTES / 16, PANEL16 = PANEL_BYTES / 16;  // descriptors count 16 bytes
  const uint32_t tmem = uniform(C.tmem), q_low = smem_descriptor_low(q_smem, 0);
  const uint32_t k_low = smem_descriptor_low(ring, 0), v_low = smem_descriptor_low(ring, PANEL_BYTES);
  Walk<NH> walk;
  walk.begin(P, C, my_tiles);
  Segment s;
  uint32_t n = 0, segment = 0, tile = 0;  // loads, segments, tiles so far
  uint32_t* status = P.L.status;

  const uint32_t id_s = uniform(P.negative ? ID_S | MMA_NEGATE_A : ID_S);
  uint32_t clean = 0;  // bit i: parity of slot i's next cleaning

  auto scores = [&](int h, uint32_t stage) {
    const uint32_t a = uniform(q_low) + h * KV16, b = uniform(k_low + stage * KV16);
    if (elect()) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int at = (k / 4) * PANEL16 + (k % 4) * 2;
        mma_ss(tmem + h * TILE, smem_descriptor(a + at), smem_descriptor(b + at), id_s, k > 0);
      }
      mma_commit(&C.s_full[h]);
    }
    __syncwarp();
  };

  while (walk.next(P, s)) {
    const uint32_t ks = n % Y::STAGES;
    if (!warp_wait(&C.q_full, segment & 1, C, status)) return false;
    if (!warp_wait(&C.full[ks], (n / Y::STAGES) & 1, C, status)) return false;
    tmem_fence_after();
    for (int h = 0; h < NH; ++h) scores(h, ks);
    if (elect()) {
      mma_commit(&C.empty[ks]);
      if (s.first + 1 == s.last) mma_commit(&C.q_empty);
    }
    __syncwarp();
    for (int t = s.first; t < s.last; ++t, n += 2, ++tile) {
      const uint32_t vs = (n + 1) % Y::STAGES, next = (n + 2) % Y::STAGES;
      const uint32_t b = uniform(v_low + vs * KV16), add = uniform(t > s.first);
      const bool more = t + 1 < s.last;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h == 0) {
          if (!warp_wait(&C.full[vs], ((n + 1) / Y::STAGES) & 1, C, status)) return false;
          if ((t + 1) * TILE > s.clear) {
            if (!warp_wait(&C.clean[vs], (clean >> vs) & 1, C, status)) return false;
            clean ^= 1u << vs;
          }
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (!warp_wait(&C.w_full[h][part], tile & 1, C, status)) return false;
          tmem_fence_after();
          if (elect()) {
#pragma unroll
            for (int k = part * TILE / 32; k < (part + 1) * TILE / 32; ++k)
              mma_ts(tmem + NH * TILE + h * D, tmem + h * TILE + k * 8, smem_descriptor(b + k * (16 * 128 / 16)), ID_O,
                     k > 0 || add);
            if (part == 1 && !more) mma_commit(&C.o_full[h]);
          }
          __syncwarp();
        }
        if (more) {
          if (h == 0 && !warp_wait(&C.full[next], ((n + 2) / Y::STAGES) & 1, C, status)) return false;
          tmem_fence_after();
          scores(h, next);
        }
      }
      if (elect()) {
        mma_commit(&C.empty[vs]);
        if (more) mma_commit(&C.empty[next]);
        if (t + 2 == s.last) mma_commit(&C.q_empty);
      }
      __syncwarp();
    }
    ++segment;
  }
  return true;
}

// Two warps, ahead of the softmax: an item's queries and its nodes' parents
// into shared memory, and the values of tiles that not every row sees whole:
// those past the item's end and those that are not finite become zeros.
template <typename T, int D, int NH>
__device__ __forceinline__ void side_role(const Plan& P, Control& C, uint32_t q_smem, uint8_t* ring, int64_t my_tiles) {
  using Y = Layout<D, NH>;
  constexpr int CHUNKS = D / 8, THREADS = 64;
  const int t = threadIdx.x % THREADS;
  uint32_t* status = P.L.status;
  Walk<NH> walk;
  walk.begin(P, C, my_tiles);
  Segment s;
  uint32_t segment = 0, tile = 0;
  for (; walk.next(P, s); ++segment, tile += s.last - s.first) {
    const Rows rows(P, s.row0);
    if (!warp_wait(&C.q_empty, (segment & 1) ^ 1, C, status)) return;
    const int n = min(NH * TILE, P.rows - s.row0), ch = t % CHUNKS;
    const T* from = static_cast<const T*>(P.L.q.data) + s.b * P.L.q.tree_stride +
                    static_cast<int64_t>(s.head) * P.group * P.L.q.head_stride + ch * 8;
    for (int r = t / CHUNKS; r < n; r += THREADS / CHUNKS) {
      int i, g;
      rows.get(P, r, i, g);
      const bool live = P.L.nodes.begin + i < s.cnt;
      async_copy16(q_smem + (r / TILE) * Y::KV_BYTES + (ch / 8) * PANEL_BYTES + (r % TILE) * 128 + (((ch % 8) ^ (r % 8)) * 16),
                   live ? from + i * P.L.q.node_stride + g * P.L.q.head_stride : from, !live);
    }
    if (P.L.nodes.parent) {
      for (int i = t; i < s.cnt; i += THREADS) {
        const int up = P.L.nodes.parent[static_cast<int64_t>(s.b) * P.L.nodes.stride + i];
        C.parent[segment % 2][i] = static_cast<uint16_t>(up < 0 || up >= i ? 0xffff : up);
        if (up >= i) set_status(status, SPEC_TREE_S_NODES);
      }
    }
    async_copies_wait();
    fence_proxy_async_smem();
    warp_arrive(&C.q_full);

    const int first_masked = s.clear / TILE;
    for (int j = max(s.first, first_masked); j < s.last; ++j) {
      const uint32_t v = 2 * (tile + j - s.first) + 1;
      if (!warp_wait(&C.full[v % Y::STAGES], (v / Y::STAGES) & 1, C, status)) return;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int row = part * 64 + t;  // a token
        uint8_t* at = ring + (v % Y::STAGES) * Y::KV_BYTES + row * 128;
        const bool past = j * TILE + row >= s.end;
        bool odd = false;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          uint4* w4 = reinterpret_cast<uint4*>(at + (c / 8) * PANEL_BYTES + (((c % 8) ^ (row % 8)) * 16));
          if (past) {
            *w4 = make_uint4(0, 0, 0, 0);
          } else {
            const uint4 x = *w4;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool lo = odd16<T>(w[e]), hi = odd16<T>(w[e] >> 16);
              if (lo) w[e] &= 0xffff0000u;
              if (hi) w[e] &= 0x0000ffffu;
              hit |= lo || hi;
            }
            if (hit) *w4 = make_uint4(w[0], w[1], w[2], w[3]);
            odd |= hit;
          }
        }
        const uint32_t word = __ballot_sync(FULL, odd);
        if (t % 32 == 0) C.odd[segment % 3][(j - first_masked) * (TILE / 32) + part * 2 + t / 32] = word;
      }
      fence_proxy_async_smem();
      warp_arrive(&C.clean[v % Y::STAGES]);
    }
  }
}

// 128 threads, one row each: weights, the running reference and sum, and the
// output.
template <typename T, int D, int NH>
__device__ __forceinline__ void softmax_role(const Plan& P, Control& C, int64_t my_tiles, int cta, int ctas, int half) {
  constexpr float SHIFT = std::is_same<T, __half>::value ? 7.0f : 0.0f;
  const int t = threadIdx.x % TILE, warp = t / 32;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t tm_s = C.tmem + half * TILE + lanes, tm_o = C.tmem + NH * TILE + half * D + lanes;
  uint32_t* status = P.L.status;
  Walk<NH> walk;
  walk.begin(P, C, my_tiles);
  Segment s;
  uint32_t tile = 0, segment = 0;
  bool ok = true;  // uniform over the warp
  for (; walk.next(P, s); ++segment) {
    const int local = half * TILE + t, row = s.row0 + local;
    int i, g;
    Rows(P, s.row0).get(P, local, i, g);
    const int node = P.L.nodes.begin + i;
    const bool live = row < P.rows && node < s.cnt;
    const bool warp_live = __any_sync(FULL, live);
    const int first_masked = s.clear / TILE;  // tiles from here on are not seen whole by every row
    float ref = -INFINITY, sum = 0.0f;

    for (int j = s.first; j < s.last; ++j, ++tile) {
      const int base = j * TILE;
      const bool masked = base + TILE > s.clear;
      ok = ok && warp_wait(&C.s_full[half], tile & 1, C, status);
      if (warp_live && ok) {
        tmem_fence_after();
        uint32_t x[TILE];
#pragma unroll
        for (int c = 0; c < TILE / 32; ++c) tmem_ld32(tm_s + c * 32, x + c * 32);
        tmem_wait_ld();
        if (masked) {
          const uint16_t* parent = C.parent[segment % 2];
          const Seen v = seen_of(P, s, live ? node : -1, base, [&](int n) { return parent[n] == 0xffff ? -1 : parent[n]; });
#pragma unroll
          for (int c = 0; c < TILE; ++c)
            if (!((v.w[c / 32] >> (c % 32)) & 1)) x[c] = 0xff800000u;
        }
        float top8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) top8[c] = fmaxf(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
#pragma unroll
        for (int c = 16; c < TILE; c += 2)
          top8[c / 2 % 8] = max3(top8[c / 2 % 8], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        const float top = P.scale2 * fmaxf(max3(max3(top8[0], top8[1], top8[2]), top8[3], top8[4]),
                                           max3(top8[5], top8[6], top8[7]));
        const bool grow = live && top > ref + LAZY;
        if (j == s.first) {
          ref = top;
        } else if (__any_sync(FULL, grow)) {
          const float f = grow ? ex2(ref - top) : 1.0f;
          if (grow) ref = top;
          sum *= f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tm_o + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tm_o + c * 32, o);
          }
        }
        const float sub = ref == -INFINITY ? 0.0f : ref - SHIFT;
        const F2 scale2(P.scale2, P.scale2), shift2(-sub, -sub);
        F2 part[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) part[c] = F2(0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // the product starts on the first half of the weights
#pragma unroll
          for (int c = p * TILE / 2; c < (p + 1) * TILE / 2; c += 2) {
            float a, b;
            fma2(F2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), scale2, shift2).get(a, b);
            a = ex2(a);
            b = ex2(b);
            part[c / 2 % 4] = add2(part[c / 2 % 4], F2(a, b));
            x[c / 2] = Pair<T>::pack(a, b);
          }
          tmem_st32(tm_s + p * 32, x + p * 32);
          tmem_wait_st();
          tmem_fence_before();
          if (p == 0) warp_arrive(&C.w_full[half][0]);
        }
        float a, b;
        add2(add2(part[0], part[1]), add2(part[2], part[3])).get(a, b);
        sum += a + b;
      } else {
        warp_arrive(&C.w_full[half][0]);
      }
      warp_arrive(&C.w_full[half][1]);
    }

    ok = ok && warp_wait(&C.o_full[half], segment & 1, C, status);
    if (!ok || s.row0 + half * TILE + warp * 32 >= P.rows) continue;
    tmem_fence_after();
    const bool whole = s.first == 0 && s.last == s.tiles;
    const Workspace ws = workspace_of(P.L.workspace, P.L.num_sms, P.ws_rows);
    const int64_t part = cta * 2 + (s.first == 0 ? 1 : 0);
    const bool some = live && sum != 0.0f;
    const float inv = some ? 1.0f / sum : 0.0f;
    uint32_t odd = 0;
    for (int j = max(s.first, first_masked); j < s.last; ++j)
      for (int e = 0; e < TILE / 32; ++e) odd |= C.odd[segment % 3][(j - first_masked) * (TILE / 32) + e];
    T* out = static_cast<T*>(P.L.out.data) + s.b * P.L.out.tree_stride + i * P.L.out.node_stride +
             (static_cast<int64_t>(s.head) * P.group + g) * P.L.out.head_stride;
    float4* partial = ws.out + part * (D / 4) * P.ws_rows + local;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      __syncwarp();
      tmem_ld32(tm_o + c * 32, o);
      tmem_wait_ld();
      if (odd && live) {  // rare: what the zeros in the values' place have left out
        for (int j = max(s.first, first_masked); j < s.last; ++j) {
          const int32_t* parent = P.L.nodes.parent + static_cast<int64_t>(s.b) * P.L.nodes.stride;
          const Seen v = seen_of(P, s, node, j * TILE, [&](int n) { return parent[n] < n ? parent[n] : -1; });
          for (int e = 0; e < TILE; ++e) {
            if (!((C.odd[segment % 3][(j - first_masked) * (TILE / 32) + e / 32] >> (e % 32)) & 1)) continue;
            uint32_t word = v.w[0];
#pragma unroll
            for (int k = 1; k < TILE / 32; ++k)
              if (e / 32 == k) word = v.w[k];
            if (!((word >> (e % 32)) & 1)) continue;
            const int64_t off = kv_slot_offset(P.L.kv, s.b, j * TILE + e, P.page_shift);
            if (off < 0) continue;
            const T* from = static_cast<const T*>(P.L.kv.v) + P.L.layer * P.L.kv.layer_stride + off +
                            s.head * P.L.kv.head_stride + c * 32;
#pragma unroll
            for (int d = 0; d < 32; ++d) {
              const float x = static_cast<float>(from[d]);
              if (!isfinite(x)) o[d] = __float_as_uint(__uint_as_float(o[d]) + x);
            }
          }
        }
      }
      if (!whole) {
        if (live) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            partial[(c * 8 + q) * P.ws_rows] = make_float4(__uint_as_float(o[q * 4]), __uint_as_float(o[q * 4 + 1]),
                                                           __uint_as_float(o[q * 4 + 2]), __uint_as_float(o[q * 4 + 3]));
        }
      } else if (row < P.rows) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = some ? __uint_as_float(o[q * 8 + e]) * inv : 0.0f;
          *reinterpret_cast<uint4*>(out + c * 32 + q * 8) = pack8<T>(y);
        }
      }
    }
    if (!whole && live) ws.sums[part * P.ws_rows + local] = make_float2(ref, sum);
    tmem_fence_before();
    if (!whole && s.first == 0 && local == 0) {
      // the CTAs after this one whose ranges begin inside the item
      const int64_t end = range_start(C.total, cta + 1, ctas) + (s.tiles - s.last);
      int pieces = 1;
      while (cta + pieces < ctas && range_start(C.total, cta + pieces, ctas) < end) ++pieces;
      ws.records[cta] = JoinRecord{pieces, s.b, s.row0, s.head};
    }
  }
}

template <typename T, int D, int NH>
__global__ void __launch_bounds__(Layout<D, NH>::THREADS, 1)
    attend_kernel(const __grid_constant__ Plan P, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Y = Layout<D, NH>;
  extern __shared__ __align__(1024) uint8_t smem[];  // nothing static, so it starts on a swizzle group
  uint8_t* ring = smem + Y::Q_BYTES;
  Control& C = *reinterpret_cast<Control*>(ring + Y::STAGES * Y::KV_BYTES);
  const int warp = __shfl_sync(FULL, threadIdx.x / 32, 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < Y::STAGES; ++i) {
      mbar_init(&C.full[i], 1);
      mbar_init(&C.empty[i], 1);
      mbar_init(&C.clean[i], 2);
    }
    mbar_init(&C.q_full, 2);
    mbar_init(&C.q_empty, 1);
    mbar_init(&C.drain, 1);
    for (int h = 0; h < NH; ++h) {
      mbar_init(&C.s_full[h], 1);
      mbar_init(&C.w_full[h][0], 4);
      mbar_init(&C.w_full[h][1], 4);
      mbar_init(&C.o_full[h], 1);
    }
    C.abort = 0;
    fence_mbar_init();
  }
  if (warp == NH * 4) tmem_alloc(&C.tmem, Y::COLUMNS);
  tmem_fence_before();
  grid_dependency_wait();
  grid_dependents_launch();

  // where this CTA's range begins: a scan of the trees' tiles
  const int B = P.L.B, per = (B + Y::THREADS - 1) / Y::THREADS;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += tree_tiles<NH>(P, b);
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(FULL, before, o);
    if (threadIdx.x % 32 >= o) before += up;
  }
  if (threadIdx.x % 32 == 31) C.scan[warp] = before;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < Y::THREADS / 32; ++w) {
    if (w < warp) before += C.scan[w];
    total += C.scan[w];
  }
  before -= mine;
  const int ctas = static_cast<int>(min64(gridDim.x, total)), cta = blockIdx.x;
  const int64_t from = range_start(total, min(cta, ctas), ctas), to = range_start(total, min(cta + 1, ctas), ctas);
  if (from < to && before <= from && from < before + mine) {
    int64_t at = before;
    for (int b = b0; b < b1; ++b) {
      const int64_t n = tree_tiles<NH>(P, b);
      if (from < at + n) {
        int64_t skip = from - at;
        int len, cnt;
        tree_of(P, b, len, cnt);
        for (int rt = 0;; ++rt) {
          int end, tiles;
          item_tiles<NH>(P, len, cnt, rt, end, tiles);
          const int64_t all = static_cast<int64_t>(tiles) * P.L.kv.n_kv_heads;
          if (skip < all) {
            C.b = b;
            C.rt = rt;
            C.head = static_cast<int>(skip / tiles);
            C.at = static_cast<int>(skip % tiles);
            break;
          }
          skip -= all;
        }
        break;
      }
      at += n;
    }
  }
  if (threadIdx.x == 0) {
    C.total = total;
    workspace_of(P.L.workspace, P.L.num_sms, P.ws_rows).records[cta].pieces = 0;
  }
  if (cta == 0)
    for (int b = threadIdx.x; b < B; b += Y::THREADS) {
      int len, cnt;
      if (const uint32_t bad = tree_of(P, b, len, cnt)) set_status(P.L.status, bad);
    }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();

  // a softmax thread holds a row of 128 scores in registers: with two halves
  // (384 threads of 168 registers) the helpers give some of theirs up
  if (NH > 1) {
    if (warp < NH * 4)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  }
  if (warp < NH * 4) {
    softmax_role<T, D, NH>(P, C, to - from, cta, ctas, warp / 4);
  } else if (warp == NH * 4) {
    load_role<D, NH>(P, &mk, &mv, C, smem_u32(ring), to - from);
  } else if (warp == NH * 4 + 1) {
    if (!product_role<T, D, NH>(P, C, smem_u32(smem), smem_u32(ring), to - from)) {
      if (elect()) mma_commit(&C.drain);  // products in flight end before their memory is given back
      mbar_wait(&C.drain, 0);
    }
  } else {
    side_role<T, D, NH>(P, C, smem_u32(smem), ring, to - from);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == NH * 4) {
    tmem_fence_after();
    tmem_free(C.tmem, Y::COLUMNS);
  }
}

// The rows of items whose tiles lie in several ranges: CTA x of grid.x looks
// at what range x left, one thread per 8 elements of a row.
constexpr int JOIN_THREADS = 256;

template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) attend_join_kernel(const __grid_constant__ Plan P) {
  grid_dependency_wait();
  grid_dependents_launch();
  const Workspace ws = workspace_of(P.L.workspace, P.L.num_sms, P.ws_rows);
  const int cta = blockIdx.x;
  const JoinRecord rec = ws.records[cta];
  const int idx = blockIdx.y * JOIN_THREADS + threadIdx.x, r = idx % P.ws_rows, q = idx / P.ws_rows;
  if (rec.pieces == 0 || q >= D / 8 || rec.row0 + r >= P.rows) return;
  int i, g;
  Rows(P, rec.row0).get(P, r, i, g);
  int len, cnt;
  tree_of(P, rec.b, len, cnt);
  float y[8], sum = 0.0f, top = -INFINITY;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.0f;
  if (P.L.nodes.begin + i < cnt) {
    // part p of the item: the end of range cta, then the starts of the next ones
    auto part = [&](int p) { return static_cast<int64_t>(cta + p) * 2 + (p == 0 ? 1 : 0); };
#pragma unroll 4
    for (int p = 0; p < rec.pieces; ++p) top = fmaxf(top, ws.sums[part(p) * P.ws_rows + r].x);
    const float sub = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
    for (int p = 0; p < rec.pieces; ++p) {
      const float2 ms = ws.sums[part(p) * P.ws_rows + r];
      const float4* o = ws.out + (part(p) * (D / 4) + q * 2) * P.ws_rows + r;
      const float4 a = o[0], b = o[P.ws_rows];
      const float f = ex2(ms.x - sub);
      sum += ms.y * f;
      y[0] += a.x * f, y[1] += a.y * f, y[2] += a.z * f, y[3] += a.w * f;
      y[4] += b.x * f, y[5] += b.y * f, y[6] += b.z * f, y[7] += b.w * f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = sum == 0.0f ? 0.0f : y[e] / sum;
  T* out = static_cast<T*>(P.L.out.data) + rec.b * P.L.out.tree_stride + i * P.L.out.node_stride +
           (static_cast<int64_t>(rec.head) * P.group + g) * P.L.out.head_stride + q * 8;
  *reinterpret_cast<uint4*>(out) = pack8<T>(y);
}

// -------------------------------------------------------------------- host ---

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &res) == cudaSuccess &&
        res == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

// [page][head][token][element] of one layer: boxes of `box` tokens of 64
// elements, one head, one page.
bool pool_map(CUtensorMap* map, const spec_tree_kv_t& kv, void* base, int layer, int box) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(kv.page_size),
                              static_cast<cuuint64_t>(kv.n_kv_heads), static_cast<cuuint64_t>(kv.n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kv.token_stride) * 2, static_cast<cuuint64_t>(kv.head_stride) * 2,
                                 static_cast<cuuint64_t>(kv.page_stride) * 2};
  const cuuint32_t boxes[4] = {PANEL, static_cast<cuuint32_t>(box), 1, 1}, steps[4] = {1, 1, 1, 1};
  return fn(map, kv.dtype == SPEC_TREE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            static_cast<uint16_t*>(base) + layer * kv.layer_stride, dims, strides, boxes, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int NH>
cudaError_t attend(Plan& P, cudaStream_t stream) {
  using Y = Layout<D, NH>;
  constexpr int SMEM = Y::Q_BYTES + Y::STAGES * Y::KV_BYTES + static_cast<int>(sizeof(Control));
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static_assert(NH * (TILE + D) <= Y::COLUMNS, "tensor memory");
  P.row_tiles = (P.rows + NH * TILE - 1) / (NH * TILE);
  CUtensorMap mk, mv;
  if (!pool_map(&mk, P.L.kv, P.L.kv.k, P.L.layer, P.box) || !pool_map(&mv, P.L.kv, P.L.kv.v, P.L.layer, P.box))
    return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(attend_kernel<T, D, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (err != cudaSuccess) return err;
  err = launch_pdl(attend_kernel<T, D, NH>, dim3(P.L.num_sms), dim3(Y::THREADS), SMEM, stream, P, mk, mv);
  if (err != cudaSuccess) return err;
  return launch_pdl(attend_join_kernel<T, D>, dim3(P.L.num_sms, (P.ws_rows * (D / 8) + JOIN_THREADS - 1) / JOIN_THREADS),
                    dim3(JOIN_THREADS), 0, stream, P);
}

template <typename T, int D>
cudaError_t attend_rows(Plan& P, cudaStream_t stream) {
  return P.rows > TILE ? attend<T, D, 2>(P, stream) : attend<T, D, 1>(P, stream);
}

int workspace_rows(int64_t rows) { return static_cast<int>(min64(rows, 2 * TILE)); }

}  // namespace

size_t attend_workspace_bytes(int num_sms, int64_t rows, int head_dim) {
  const Workspace w = workspace_of(nullptr, num_sms, workspace_rows(rows));
  return reinterpret_cast<size_t>(w.out) + static_cast<size_t>(num_sms) * 2 * workspace_rows(rows) * head_dim * 4;
}

cudaError_t launch_attend(const AttendLaunch& L, cudaStream_t stream) {
  Plan P;
  P.L = L;
  P.group = L.n_q_heads / L.kv.n_kv_heads;
  P.rows = L.nodes.count * P.group;
  P.page_shift = log2_of(L.kv.page_size);
  P.box = L.kv.page_size < TILE ? L.kv.page_size : TILE;
  P.ws_rows = workspace_rows(P.rows);
  // a scale of zero would turn -inf into NaN: weights 2^(1e-30 S) are all one as well
  P.scale2 = fminf(fmaxf(fabsf(L.scale) * 1.4426950408889634f, 1e-30f), 3e38f);
  P.negative = L.scale < 0.0f;
  P.group_inv = P.group == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + P.group - 1) / P.group);
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend_rows<__nv_bfloat16, 128>(P, stream) : attend_rows<__nv_bfloat16, 64>(P, stream);
  return L.kv.head_dim == 128 ? attend_rows<__half, 128>(P, stream) : attend_rows<__half, 64>(P, stream);
}

}  // namespace st
