// Attention of a tree's nodes over a paged key-value cache (spec_tree_attend).
//
// Rows.  The query heads that share a key head, over all nodes of the call,
// are the rows of one product: row r is node r / group, head r % group.  The
// rows of as many whole nodes as 128 lanes have room for fill one accumulator
// ("half"); a CTA has two, so that one half's softmax runs under the other
// half's products:
//   - calls of more rows than a half's take two halves' at a time and load keys
//     and values once for both;
//   - calls of no more (PAIR) give both halves the same rows: one takes
//     the even tiles of a segment, the other the odd ones, and their sums are
//     put together at its end.
//
// Work.  An item is (tree, one or two halves' rows, key head); its tokens are cut
// into tiles of 128.  The tiles are dealt to the CTAs (one per SM) in one of
// two ways:
//   - ranges: all items' tiles, one after the other, in equal consecutive
//     ranges.  A long cache is split over the card and a ragged batch is
//     balanced; a CTA begins and ends inside items;
//   - pieces, where the items are fewer than the CTAs: each item cut into
//     equal pieces, one per CTA, their length the least of 32 tried for which
//     there are CTAs enough (find_piece).  Taken where the length and one
//     segment's fixed cost are below a range's length and two.
// An item that one CTA has whole is finished there; otherwise each CTA leaves
// its sums, their reference and its unnormalised output in the workspace, and
// the parts are put together in the item's order:
//   - ranges: an item is what its first CTA does last and the next ones do
//     first, so the others have nearly always left their parts when the first
//     comes to its own, and it puts them together without leaving its own.  If
//     not, and for calls of up to 16 rows, whoever is the last to leave a part
//     does it;
//   - pieces, of more rows: they end together, and one CTA would be long about
//     it: attend_join_kernel, over all SMs.  It is launched behind every call that
//     may be dealt in pieces, as the lengths are known on the device alone.
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
// NaN among the values are replaced by zero in shared memory first.
//
// Values that are not finite.  A seen one counts whatever its weight: an element
// of a row's output is the sum of the seen values there that are not finite, if
// there are any.  The products say no more than that there are some: a weight or
// a rescaling that is zero in its few bits makes NaN of an infinity.  So a row
// whose output is not finite though its weights are has the segment's values
// read again (settle), each part of an item carries its own sum, and the join
// adds those of the parts (settle_joined).  Where all is finite that costs a
// product with zero per element of the output: 0.2 to 0.5 us of 10 to 38 us where
// segments are few (one token of one short sequence 9.7 -> 10.1, frontier 34.9 ->
// 35.5, 32 key heads 37.3 -> 37.6), nothing where they are many.  With an infinity
// in every page, calls take 4 to 10 times as long (one token of 64 sequences 166
// -> 1610 us, 8 trees 38 -> 141); where all elements are NaN the reading stops.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <atomic>
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
constexpr int MAX_SLOTS = 5;                    // of a ring
constexpr int MASKED_TILES = SPEC_TREE_MAX_NODES / TILE + 2;
constexpr float LAZY = 8.0f;                    // log2 of what a weight may exceed its reference by
constexpr int THREADS = 3 * TILE;               // two softmax warpgroups and one of helpers
constexpr int HELPERS = 2 * TILE / 32;          // the helpers' first warp
constexpr int COLUMNS = 512;                    // tensor memory: S of both halves, then O of both
constexpr int MAX_PIECE_ITEMS = 256;            // (tree, rows) of calls that may be dealt in pieces
constexpr int JOIN_PARTS = 4;                   // parts of an item joined at a time
// Rows of calls that need no join kernel.  By the last CTA to come, and by the
// kernel: 4 rows, one sequence of 500 tokens 9.9 and 11.4 us, of 16384 19.8 and
// 21.5, 4 of 4000 16.5 and 18.0; 32 rows over 8192 25.0 and 20.0; 244 rows over
// 8192 46.0 and 34.4.  Many parts are the exception: one warp walks them, four at
// a time, and 8 rows over 16384 tokens of one key head (129 parts) take 54.4 and
// 46.0.
constexpr int JOIN_INSIDE_ROWS = 16;
// Weights are handed to the product in two parts, so that it works on the first
// while the second is made.
constexpr int EARLY = 64;

struct Plan {
  AttendLaunch L;
  int group, rows, half_rows, row_tiles, page_shift, box, ws_rows;
  uint64_t group_inv;  // floor(2^64 / group) + 1, 0 for a group of one
  float scale2;        // |scale| log2(e)
  bool may_piece;      // no more items than CTAs
  bool negative;       // scale < 0: the products take -Q
  bool join_inside;    // no join kernel
  int q_box;           // nodes of a copy of queries
};

struct JoinRecord {
  int32_t parts, b, row0, head;  // parts = 0: nothing to join
};

// Parts of items: slot 0 of a CTA for one that began before it, slot 1 for one
// that goes on after it.
struct Workspace {
  uint32_t* arrived;    // [CTA where the item begins][softmax warp]: parts left; zero between calls
  JoinRecord* records;  // [CTA]: the item of which it has the first piece, for the join kernel
  float2* sums;         // [CTA][2][ws_rows]: (reference, sum)
  float4* out;          // [CTA][2][D / 4][ws_rows]: neighbouring rows are neighbours in memory
};

__host__ __device__ inline Workspace workspace_of(void* ws, int num_sms, int ws_rows) {
  Workspace w;
  w.arrived = static_cast<uint32_t*>(ws);
  w.records = reinterpret_cast<JoinRecord*>(w.arrived + num_sms * 8);
  w.sums = reinterpret_cast<float2*>(w.records + num_sms);
  w.out = reinterpret_cast<float4*>(w.sums + static_cast<size_t>(num_sms) * 2 * ws_rows);
  return w;
}

template <int D, bool PAIR>
struct Layout {
  static constexpr int HALVES = PAIR ? 1 : 2;  // of an item's rows
  static constexpr int PANELS = D / PANEL;
  static constexpr int KV_BYTES = PANELS * PANEL_BYTES;
  static constexpr int Q_BYTES = HALVES * KV_BYTES;
  // tiles that the rings of keys and of values hold: what 7 * 32 KB leave
  static constexpr int SLOTS = (7 * 32768 - Q_BYTES) / KV_BYTES;
  static constexpr int KS = (SLOTS + 1) / 2 < MAX_SLOTS ? (SLOTS + 1) / 2 : MAX_SLOTS;
  static constexpr int VS = SLOTS / 2 < MAX_SLOTS ? SLOTS / 2 : MAX_SLOTS;
};

// A consecutive piece of an item's tiles: what one CTA does at a time.
struct Segment {
  int b, rt, head, row0;   // row0: first row of the item
  int len, cnt;            // committed tokens, nodes that exist
  int first, last, tiles;  // tiles first .. last - 1 of `tiles`
  int end;                 // tokens (slots) the item reads
  int clear;               // slots below this one are seen by every row of the item
  int64_t begin;           // where the item begins among all tiles (ranges)
};

struct Control {
  uint64_t k_full[MAX_SLOTS], k_empty[MAX_SLOTS], v_full[MAX_SLOTS], v_empty[MAX_SLOTS], v_clean[MAX_SLOTS];
  uint64_t q_full, q_empty, s_full[2], w_full[2][2], o_full[2], drain;
  uint32_t tmem;
  int abort;
  int64_t scan[THREADS / 32];
  int64_t total;            // tiles of the call (ranges)
  int64_t count;            // this CTA's tiles
  int pieces, piece;        // pieces of this CTA's item (0: ranges), and which one this is
  Segment start;            // where this CTA begins
  uint32_t odd[3][MASKED_TILES * (TILE / 32)];  // tokens with a value that is not finite, by segment modulo 3
  uint8_t up[2][SPEC_TREE_MAX_NODES];           // node minus parent, by segment modulo 2; 0: none, 255: more
  union {
    float2 pair[TILE];         // the odd tiles' (reference, sum)
    int tiles[MAX_PIECE_ITEMS];  // setup: tiles of (tree, rows)
  };
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

__device__ __forceinline__ int node_of_row(const Plan& P, int row) {  // row / group
  return P.group_inv ? static_cast<int>(__umul64hi(row, P.group_inv)) : row;
}

template <int HALVES>
__device__ __forceinline__ void item_tiles(const Plan& P, int len, int cnt, int rt, int& end, int& tiles) {
  const int item_rows = HALVES * P.half_rows;
  const int last_row = min((rt + 1) * item_rows, P.rows) - 1;
  const int nodes = min(cnt, P.L.nodes.begin + node_of_row(P, last_row) + 1);
  const int first = P.L.nodes.begin + node_of_row(P, rt * item_rows);
  end = first < cnt ? len + nodes : 0;  // rows of nodes that do not exist read nothing
  tiles = end > 0 ? (end + TILE - 1) / TILE : 1;
}

// Tiles of one key head of item group x: tree x / row_tiles, rows x % row_tiles.
template <int HALVES>
__device__ __forceinline__ int group_tiles(const Plan& P, int x) {
  const int b = P.row_tiles == 1 ? x : x / P.row_tiles;
  int len, cnt, end, tiles;
  tree_of(P, b, len, cnt);
  item_tiles<HALVES>(P, len, cnt, x - b * P.row_tiles, end, tiles);
  return tiles;
}

// The item (tree s.b, rows s.rt); its lengths are there already if `known`.
template <int HALVES>
__device__ __forceinline__ void set_item(const Plan& P, Segment& s, bool known) {
  if (!known) tree_of(P, s.b, s.len, s.cnt);
  s.row0 = s.rt * HALVES * P.half_rows;
  item_tiles<HALVES>(P, s.len, s.cnt, s.rt, s.end, s.tiles);
  s.clear = P.L.nodes.parent ? s.len : s.len + min(s.cnt, P.L.nodes.begin + node_of_row(P, s.row0) + 1);
}

// Where range c of `ctas` (at most 2^8) begins, and the range that holds tile
// `at`.  64-bit divisions are long: there are seldom tiles enough for them.
__device__ __forceinline__ int64_t range_start(int64_t total, int c, int ctas) {
  if (total < 1 << 24) return static_cast<uint32_t>(total) * c / ctas;
  return total * c / ctas;
}

__device__ __forceinline__ int range_of(int64_t total, int64_t at, int ctas) {
  const int c = total < 1 << 24 ? static_cast<uint32_t>(at) * ctas / static_cast<uint32_t>(total)
                                : static_cast<int>(at * ctas / total);
  return range_start(total, c + 1, ctas) <= at ? c + 1 : c;
}

// The segments of a CTA, one after the other; every role walks them for itself.
template <int HALVES>
struct Walk {
  Segment s;
  int64_t left;
  bool fresh = true;

  __device__ __forceinline__ explicit Walk(const Control& C) : s(C.start), left(C.count) {}

  __device__ __forceinline__ bool next(const Plan& P) {
    if (left <= 0) return false;
    if (!fresh) {
      s.first = 0;
      s.begin += s.tiles;
      if (++s.head == P.L.kv.n_kv_heads) {
        s.head = 0;
        const bool same = ++s.rt < P.row_tiles;
        if (!same) s.rt = 0, ++s.b;
        set_item<HALVES>(P, s, same);
      }
    }
    fresh = false;
    const int n = static_cast<int>(min64(left, s.tiles - s.first));
    s.last = s.first + n;
    left -= n;
    return true;
  }
};

// A wait that gives up when it, or another role of the CTA, has run out.
// (The kernel's code is cold in the instruction cache when a CTA starts, so
// what is not on the way of every tile is kept out of line or rolled.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Control& C, uint32_t* status) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (uint32_t it = 0; it < WAIT_LIMIT; ++it) {
    uint32_t done;
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

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// A barrier of some of the CTA's warps (converged: .aligned instructions of a
// warp whose lanes have parted are undefined).
__device__ __forceinline__ void warps_meet(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// bit j: the row's node sees slot `base` + j of the 128 slots of a tile
struct Seen {
  uint32_t w[TILE / 32];
  __device__ __forceinline__ uint32_t get(int i) const { return i < 2 ? (i == 0 ? w[0] : w[1]) : (i == 2 ? w[2] : w[3]); }
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

// Two warps, one for keys and one for values: tokens from their pages into the
// ring.  Lane i looks up the tile's i-th page (or the one that its 128 tokens
// lie in); pages past the item's end are not read.  A copy takes 70 to 80
// cycles to issue, whoever issues it, and at 16 tokens a page a tile has 32:
// by one warp for both, 1300 cycles for 32 KB were no faster than the SM's
// share of the memory's bandwidth.
template <int D, bool PAIR, bool KEYS>
__device__ __forceinline__ void load_role(const Plan& P, const CUtensorMap* map, Control& C, uint32_t ring) {
  using Y = Layout<D, PAIR>;
  constexpr int SLOTS = KEYS ? Y::KS : Y::VS;
  uint64_t* full = KEYS ? C.k_full : C.v_full;
  uint64_t* empty = KEYS ? C.k_empty : C.v_empty;
  const int lane = threadIdx.x % 32;
  const int boxes = TILE / P.box;
  Walk<Y::HALVES> walk(C);
  const Segment& s = walk.s;
  uint32_t n = 0;  // loads so far
  bool ok = true;
  while (ok && walk.next(P)) {
    const int32_t* table = P.L.kv.page_table + static_cast<int64_t>(s.b) * P.L.kv.table_stride;
    auto entry = [&](int t) {  // the page of this lane's copy of tile t
      const int slot = t * TILE + lane * P.box;
      return t < s.last && lane < boxes && slot < s.end ? table[slot >> P.page_shift] : 0;
    };
    int next = entry(s.first);
    for (int t = s.first; t < s.last; ++t, ++n) {
      int page = next;
      next = entry(t + 1);
      if (page < 0 || page >= P.L.kv.n_pages) {
        set_status(P.L.status, SPEC_TREE_S_PAGES);
        page = P.L.kv.n_pages;  // outside the pool: the copy fills zeros
      }
      const int off = uniform(P.box == TILE ? (t * TILE) & (P.L.kv.page_size - 1) : 0);
      const int used = s.end > 0 ? min(boxes, (s.end - t * TILE + P.box - 1) / P.box) : 0;
      const int slot = n % SLOTS;
      ok = warp_wait(&empty[slot], ((n / SLOTS) & 1) ^ 1, C, P.L.status);
      if (!ok) break;
      if (elect()) mbar_expect_tx(&full[slot], used * P.box * 128 * Y::PANELS);
      const uint32_t to = uniform(ring + slot * Y::KV_BYTES), head = uniform(s.head);
#pragma unroll 1
      for (int x0 = 0; x0 < used; x0 += 4) {
        uint32_t pages[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) pages[x] = __shfl_sync(FULL, page, x0 + x);
        if (elect()) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (x0 + x < used) {
#pragma unroll
              for (int p = 0; p < Y::PANELS; ++p)
                tile_g2s(to + p * PANEL_BYTES + (x0 + x) * P.box * 128, map, p * PANEL, off, head, pages[x], &full[slot]);
            }
        }
        __syncwarp();
      }
    }
  }
  // copies in flight land before the CTA ends, whichever role has given up (if
  // none has, the products have waited for them)
  for (uint32_t o = n > SLOTS ? n - SLOTS : 0; o < n; ++o) mbar_wait(&full[o % SLOTS], (o / SLOTS) & 1);
}

// One warp: the products.  The halves take turns, so that while one half's
// weights are made the other half's products run.  It ends early where a wait gives up.
template <typename T, int D, bool PAIR>
__device__ __forceinline__ void product_role(const Plan& P, Control& C, uint32_t q_smem, uint32_t k_smem, uint32_t v_smem) {
  using Y = Layout<D, PAIR>;
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t ID_S = mma_descriptor(BF, TILE, false), ID_O = mma_descriptor(BF, D, true);
  constexpr int KV16 = Y::KV_BYTES / 16, PANEL16 = PANEL_BYTES / 16;  // descriptors count 16 bytes
  const uint32_t tmem = uniform(C.tmem), q_low = uniform(smem_descriptor_low(q_smem, 0));
  const uint32_t k_low = smem_descriptor_low(k_smem, 0), v_low = smem_descriptor_low(v_smem, PANEL_BYTES);
  const uint32_t id_s = uniform(P.negative ? ID_S | MMA_NEGATE_A : ID_S);
  uint32_t* status = P.L.status;
  Walk<Y::HALVES> walk(C);
  const Segment& s = walk.s;
  uint32_t n = 0, segment = 0;   // tiles, segments so far
  uint32_t parity = 0;           // bit h: parity of half h's next weights
  uint32_t clean = 0;            // bit i: parity of slot i's next cleaning

  auto issue_scores = [&](uint32_t to, uint32_t a, uint32_t b, uint64_t* bar) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int at = (k / 4) * PANEL16 + (k % 4) * 2;
      mma_ss(to, smem_descriptor(a + at), smem_descriptor(b + at), id_s, k > 0);
    }
    mma_commit(bar);
  };
  auto keys = [&](uint32_t tile) { return warp_wait(&C.k_full[tile % Y::KS], (tile / Y::KS) & 1, C, status); };
  // S of half h from a tile's keys
  auto scores = [&](int h, uint32_t tile) {
    const uint32_t a = uniform(q_low + (PAIR ? 0 : h * KV16)), b = uniform(k_low + tile % Y::KS * KV16);
    const uint32_t to = uniform(tmem + h * TILE);
    if (elect()) issue_scores(to, a, b, &C.s_full[h]);
    __syncwarp();
  };
  auto give_back = [&](uint64_t* bar) {
    if (elect()) mma_commit(bar);
    __syncwarp();
  };
  // O of half h from a tile's values, as the weights' two parts come, and,
  // unless PAIR, right behind it S from the next tile's keys (which are then
  // there) if there is one; the values are given back in between
  auto output = [&](int h, uint32_t tile, bool first, bool last) {
    const uint32_t b = uniform(v_low + tile % Y::VS * KV16), add = uniform(!first), more = uniform(!last);
    const uint32_t to = uniform(tmem + 2 * TILE + h * D), from = uniform(tmem + h * TILE);
    const uint32_t qa = uniform(q_low + (PAIR ? 0 : h * KV16)), kb = uniform(k_low + (tile + 1) % Y::KS * KV16);
    if (!warp_wait(&C.w_full[h][0], (parity >> h) & 1, C, status)) return false;
    tmem_fence_after();
    if (elect()) {
#pragma unroll
      for (int x = 0; x < EARLY / 16; ++x)
        mma_ts(to, from + x * 8, smem_descriptor(b + x * (16 * 128 / 16)), ID_O, x > 0 || add);
    }
    __syncwarp();
    if (!warp_wait(&C.w_full[h][1], (parity >> h) & 1, C, status)) return false;
    tmem_fence_after();
    if (elect()) {
#pragma unroll
      for (int x = EARLY / 16; x < TILE / 16; ++x)
        mma_ts(to, from + x * 8, smem_descriptor(b + x * (16 * 128 / 16)), ID_O, true);
      if (PAIR || h == 1) mma_commit(&C.v_empty[tile % Y::VS]);
      if (!more)
        mma_commit(&C.o_full[h]);
      else if (!PAIR)
        issue_scores(from, qa, kb, &C.s_full[h]);
    }
    __syncwarp();
    parity ^= 1u << h;
    return true;
  };
  // a tile's values (token tile t), cleaned where not every row sees it whole
  auto values = [&](int t, uint32_t tile) {
    const uint32_t vs = tile % Y::VS;
    if (!warp_wait(&C.v_full[vs], (tile / Y::VS) & 1, C, status)) return false;
    if ((t + 1) * TILE > s.clear) {
      if (!warp_wait(&C.v_clean[vs], (clean >> vs) & 1, C, status)) return false;
      clean ^= 1u << vs;
    }
    return true;
  };

  while (walk.next(P)) {
    const int count = s.last - s.first;
    if (!warp_wait(&C.q_full, segment & 1, C, status) || !keys(n)) return;
    tmem_fence_after();
#pragma unroll 1
    for (int h = 0; h < 2 && (!PAIR || h < count); ++h) {
      if (PAIR && h == 1 && !keys(n + 1)) return;
      scores(h, PAIR ? n + h : n);
      if (PAIR) give_back(&C.k_empty[(n + h) % Y::KS]);
    }
    if (!PAIR) give_back(&C.k_empty[n % Y::KS]);
    if (count <= (PAIR ? 2 : 1)) give_back(&C.q_empty);
    if (PAIR) {
      // tile x by half x % 2; its successor there is tile x + 2
#pragma unroll 1
      for (int x = 0; x < count; ++x) {
        const bool more = x + 2 < count;
        if (!values(s.first + x, n + x) || !output(x & 1, n + x, x < 2, !more)) return;
        if (more) {
          if (!keys(n + x + 2)) return;
          tmem_fence_after();
          scores(x & 1, n + x + 2);
          give_back(&C.k_empty[(n + x + 2) % Y::KS]);
          if (x + 3 == count) give_back(&C.q_empty);
        }
      }
    } else {
#pragma unroll 1
      for (int x = 0; x < count; ++x) {
        const bool more = x + 1 < count;
        if (!values(s.first + x, n + x) || (more && !keys(n + x + 1))) return;
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
          if (!output(h, n + x, x == 0, !more)) return;
        if (more) give_back(&C.k_empty[(n + x + 1) % Y::KS]);
        if (x + 2 == count) give_back(&C.q_empty);
      }
    }
    n += count;
    ++segment;
  }
}

// Whether a 128-byte row holds an infinity or a NaN: those times zero are NaN.
// Neighbouring threads start at different chunks, as their rows share banks.
template <typename T>
__device__ __forceinline__ bool any_odd(const uint4* row, int rotate) {
  auto acc = Pair<T>::pair(0);
  const auto zero = acc;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 x = row[c ^ rotate];
    acc = __hfma2(Pair<T>::pair(x.x), zero, acc);
    acc = __hfma2(Pair<T>::pair(x.y), zero, acc);
    acc = __hfma2(Pair<T>::pair(x.z), zero, acc);
    acc = __hfma2(Pair<T>::pair(x.w), zero, acc);
  }
  return isnan(__low2float(acc)) || isnan(__high2float(acc));
}

// One warp, ahead of the softmax: an item's queries and its nodes' parents into
// shared memory, and the values of tiles that not every row sees whole: those
// past the item's end and those that are not finite become zeros.  It passes
// every slot of the values' ring, so that its waits keep to the ring's phases.
template <typename T, int D, bool PAIR>
__device__ __forceinline__ void side_role(const Plan& P, const CUtensorMap* mq, Control& C, uint32_t q_smem, uint8_t* v_ring) {
  using Y = Layout<D, PAIR>;
  constexpr int CHUNKS = D / 8;
  const int lane = threadIdx.x % 32;
  uint32_t* status = P.L.status;
  Walk<Y::HALVES> walk(C);
  const Segment& s = walk.s;
  uint32_t segment = 0, n = 0, asked = 0;  // segments, tiles, segments whose queries have been asked for so far
  bool ok = true;
  for (; ok && walk.next(P); ++segment) {
    ok = warp_wait(&C.q_empty, (segment & 1) ^ 1, C, status);
    if (!ok) break;
    const int node = node_of_row(P, s.row0);
    if (elect()) {
      mbar_expect_more(&C.q_full, Y::HALVES * Y::PANELS * P.q_box * P.group * 128);
#pragma unroll
      for (int h = 0; h < Y::HALVES; ++h)
#pragma unroll
        for (int p = 0; p < Y::PANELS; ++p)
          tile_g2s(q_smem + h * Y::KV_BYTES + p * PANEL_BYTES, mq, p * PANEL, s.head * P.group, node + h * P.q_box, s.b,
                   &C.q_full);
    }
    __syncwarp();
    if (P.L.nodes.parent) {
      const int32_t* parent = P.L.nodes.parent + static_cast<int64_t>(s.b) * P.L.nodes.stride;
#pragma unroll 2
      for (int x = lane; x < s.cnt; x += 32) {
        const int up = parent[x];
        C.up[segment % 2][x] = static_cast<uint8_t>(up < 0 || up >= x ? 0 : min(x - up, 255));
        if (up >= x) set_status(status, SPEC_TREE_S_NODES);
      }
    }
    warp_arrive(&C.q_full);
    asked = segment + 1;

    const int first_masked = s.clear / TILE;
    for (int j = s.first; j < s.last; ++j, ++n) {
      const int slot = n % Y::VS;
      ok = warp_wait(&C.v_full[slot], (n / Y::VS) & 1, C, status);
      if (!ok) break;
      if (j >= first_masked) {
#pragma unroll 1
        for (int part = 0; part < TILE / 32; ++part) {
          const int row = part * 32 + lane;  // a token
          uint8_t* at = v_ring + slot * Y::KV_BYTES + row * 128;
          bool odd = false;
          if (j * TILE + row >= s.end) {
#pragma unroll 4
            for (int c = 0; c < CHUNKS; ++c)
              *reinterpret_cast<uint4*>(at + (c / 8) * PANEL_BYTES + ((c ^ lane) % 8) * 16) = make_uint4(0, 0, 0, 0);
          } else if (j * TILE + row >= s.clear) {  // a token that some rows do not see
#pragma unroll 1
            for (int p = 0; p < Y::PANELS; ++p)
              odd |= any_odd<T>(reinterpret_cast<const uint4*>(at + p * PANEL_BYTES), lane % 8);
          }
          const uint32_t word = __ballot_sync(FULL, odd);
          if (odd) {
#pragma unroll 1
            for (int c = 0; c < CHUNKS * 4; ++c) {
              uint32_t* w = reinterpret_cast<uint32_t*>(at + (c / 32) * PANEL_BYTES) + c % 32;
              if (odd16<T>(*w)) *w &= 0xffff0000u;
              if (odd16<T>(*w >> 16)) *w &= 0x0000ffffu;
            }
          }
          if (lane == 0) C.odd[segment % 3][(j - first_masked) * (TILE / 32) + part] = word;
        }
        fence_proxy_async_smem();
        warp_arrive(&C.v_clean[slot]);
      }
      warp_arrive(&C.v_empty[slot]);
    }
  }
  if (asked > 0) mbar_wait(&C.q_full, (asked - 1) & 1);  // as load_role: queries in flight land before the CTA ends
}

// Whether some of the numbers taken are not finite: those times zero are NaN.
struct Finite {
  F2 acc[4];
  __device__ __forceinline__ Finite() {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = F2(0.0f, 0.0f);
  }
  template <int N>
  __device__ __forceinline__ void take(const uint32_t (&x)[N]) {
    const F2 zero(0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < N; e += 2)
      acc[e / 2 % 4] = fma2(F2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), zero, acc[e / 2 % 4]);
  }
  __device__ __forceinline__ bool all() const {
    float a, b;
    add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])).get(a, b);
    return !isnan(a + b);
  }
};

// A whole warp, a row each: the elements where the row sees values of the segment
// that are not finite become their sum, in what the row's thread has just written
// (`out`, or `partial` in the workspace's order) if the row `counts`.  `again`:
// values that every row sees may be among them, and are read again, 32 tokens at
// a time; the others are those that `odd` names.
template <typename T, int D>
__device__ __noinline__ void settle(const Plan& P, const Segment& s, const uint32_t* odd, bool again, bool counts, int node,
                                    T* out, float* partial) {
  const int lane = threadIdx.x % 32, first_masked = s.clear / TILE;
  const T* values = static_cast<const T*>(P.L.kv.v) + P.L.layer * P.L.kv.layer_stride + s.head * P.L.kv.head_stride;
  auto element = [&](int d) { return partial + static_cast<int64_t>(d / 4) * P.ws_rows * 4 + d % 4; };
  if (again) {
    // lane x of a token's LANES neighbouring ones has its elements 8 x .. 8 x + 7
    constexpr int LANES = D / 8;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    const int end = min(s.last * TILE, min(s.clear, s.end));
    auto place = [&](int t) { return t < end ? kv_slot_offset(P.L.kv, s.b, t, P.page_shift) : -1; };
    int64_t next = place(s.first * TILE + lane);
#pragma unroll 1
    for (int t0 = s.first * TILE; t0 < end; t0 += 32) {
      const int64_t off = next;
      uint4 w[LANES];
#pragma unroll
      for (int x = 0; x < LANES; ++x) {
        const int64_t at = __shfl_sync(FULL, off, x * (32 / LANES) + lane / LANES);
        w[x] = at < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(values + at + lane % LANES * 8);
      }
      next = place(t0 + 32 + lane);
#pragma unroll
      for (int x = 0; x < LANES; ++x) {
        float y[8];
        unpack8<T>(w[x], y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!isfinite(y[e])) sum[e] += y[e];
      }
      bool done = true;  // NaN everywhere: it stays so
#pragma unroll
      for (int e = 0; e < 8; ++e) done = done && isnan(sum[e]);
      if (__all_sync(FULL, done)) break;
    }
#pragma unroll
    for (int o = LANES; o < 32; o *= 2)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(FULL, sum[e], o);
#pragma unroll 1
    for (int x = 0; x < LANES; ++x) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = __shfl_sync(FULL, sum[e], x);
        if (!counts || y == 0.0f) continue;
        if (out)
          out[x * 8 + e] = T(y);
        else
          *element(x * 8 + e) = y;
      }
    }
  }
  if (!counts) return;
  const int32_t* parent = P.L.nodes.parent + static_cast<int64_t>(s.b) * P.L.nodes.stride;
#pragma unroll 1
  for (int j = max(s.first, first_masked); j < s.last; ++j) {
    const uint32_t* words = odd + (j - first_masked) * (TILE / 32);
    if ((words[0] | words[1] | words[2] | words[3]) == 0) continue;
    const Seen v = seen_of(P, s, node, j * TILE, [&](int n) { return parent[n] < n ? parent[n] : -1; });
    for (int w = 0; w < TILE / 32; ++w) {
      for (uint32_t left = words[w] & v.get(w); left; left &= left - 1) {
        const int64_t off = kv_slot_offset(P.L.kv, s.b, j * TILE + w * 32 + __ffs(left) - 1, P.page_shift);
        if (off < 0) continue;
#pragma unroll 1
        for (int d = 0; d < D; ++d) {
          const float x = static_cast<float>(values[off + d]);
          if (isfinite(x)) continue;
          if (out)
            out[d] = T(static_cast<float>(out[d]) + x);
          else
            *element(d) += x;
        }
      }
    }
  }
}

// The same for four elements of a row of an item in parts: those of CTA slots 0
// and 1 are `stride` apart, `first` is the first CTA's slot 0.
template <typename T>
__device__ __noinline__ void settle_joined(const float4* first, int64_t stride, int parts, T* out) {
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int p = 0; p < parts; ++p) {
    const float4 y = __ldcg(first + (p == 0 ? 1 : 2 * p) * stride);
    if (!isfinite(y.x)) sum[0] += y.x;
    if (!isfinite(y.y)) sum[1] += y.y;
    if (!isfinite(y.z)) sum[2] += y.z;
    if (!isfinite(y.w)) sum[3] += y.w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (sum[e] != 0.0f) out[e] = T(sum[e]);
}

// Rows local0 .. local0 + rows - 1 of an item from its parts, which the CTAs
// from `from` on have left: thread x of `threads` (a power of two) takes 16
// bytes at a time of the parts.
template <typename T, int D>
__device__ __forceinline__ void join_rows(const Plan& P, const Workspace& ws, const JoinRecord& rec, int cnt, int from,
                                          int local0, int rows, int x, int threads) {
  rows = min(rows, P.rows - rec.row0 - local0);
  // a thread keeps to one row; neighbours have neighbouring rows
  int spread = 1;
  while (spread < rows && spread < threads) spread *= 2;
  if (x % spread >= rows) return;
  const int local = local0 + x % spread, row = rec.row0 + local;
  const int i = node_of_row(P, row), g = row - i * P.group;
  const bool live = P.L.nodes.begin + i < cnt;
  T* out = static_cast<T*>(P.L.out.data) + rec.b * P.L.out.tree_stride + i * P.L.out.node_stride +
           (static_cast<int64_t>(rec.head) * P.group + g) * P.L.out.head_stride;
  // BATCH quads of JOIN_PARTS parts at a time: their loads are in flight together
  constexpr int BATCH = 4;
  const int step = threads / spread;
#pragma unroll 1
  for (int q0 = x / spread; q0 < D / 4; q0 += BATCH * step) {
    float4 acc[BATCH];
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < BATCH; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int p0 = 0; live && p0 < rec.parts; p0 += JOIN_PARTS) {
      float2 ms[JOIN_PARTS];
      float4 y[JOIN_PARTS][BATCH];
#pragma unroll
      for (int p = 0; p < JOIN_PARTS; ++p) {
        // part p: slot 1 of the first CTA, slot 0 of the next ones
        const int64_t slot = static_cast<int64_t>(from + p0 + p) * 2 + (p0 + p == 0 ? 1 : 0);
        const float4* part = ws.out + slot * (D / 4) * P.ws_rows + local;
        const bool there = p0 + p < rec.parts;
        ms[p] = there ? __ldcg(&ws.sums[slot * P.ws_rows + local]) : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const int q = q0 + e * step;
          y[p][e] = there && q < D / 4 ? __ldcg(part + q * P.ws_rows) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      }
      float next = top;
#pragma unroll
      for (int p = 0; p < JOIN_PARTS; ++p) next = fmaxf(next, ms[p].x);
      const float sub = next == -INFINITY ? 0.0f : next, keep = ex2(top - sub);
      top = next;
      sum *= keep;
#pragma unroll
      for (int e = 0; e < BATCH; ++e) acc[e].x *= keep, acc[e].y *= keep, acc[e].z *= keep, acc[e].w *= keep;
#pragma unroll
      for (int p = 0; p < JOIN_PARTS; ++p) {
        const float f = ex2(ms[p].x - sub);
        sum = fmaf(ms[p].y, f, sum);
#pragma unroll
        for (int e = 0; e < BATCH; ++e)
          acc[e].x = fmaf(y[p][e].x, f, acc[e].x), acc[e].y = fmaf(y[p][e].y, f, acc[e].y),
          acc[e].z = fmaf(y[p][e].z, f, acc[e].z), acc[e].w = fmaf(y[p][e].w, f, acc[e].w);
      }
    }
    const bool some = sum != 0.0f;  // else zeros, also where acc is not finite
    const float inv = some ? 1.0f / sum : 0.0f;
    uint32_t y[4 * BATCH];
#pragma unroll
    for (int e = 0; e < BATCH; ++e) {
      const int q = q0 + e * step;
      y[4 * e] = __float_as_uint(acc[e].x), y[4 * e + 1] = __float_as_uint(acc[e].y);
      y[4 * e + 2] = __float_as_uint(acc[e].z), y[4 * e + 3] = __float_as_uint(acc[e].w);
      if (q < D / 4)
        *reinterpret_cast<uint2*>(out + q * 4) = some ? make_uint2(Pair<T>::pack(acc[e].x * inv, acc[e].y * inv),
                                                                   Pair<T>::pack(acc[e].z * inv, acc[e].w * inv))
                                                      : make_uint2(0, 0);
    }
    Finite finite;
    finite.take(y);
    if (__builtin_expect(!finite.all(), 0) && some && !isnan(sum)) {
#pragma unroll 1
      for (int q = q0; q < min(q0 + BATCH * step, D / 4); q += step)
        settle_joined<T>(ws.out + (static_cast<int64_t>(from) * 2 * (D / 4) + q) * P.ws_rows + local,
                         static_cast<int64_t>(D / 4) * P.ws_rows, rec.parts, out + q * 4);
    }
  }
}

// 128 threads, one row each: weights, the running reference and sum, and the
// output.
template <typename T, int D, bool PAIR>
__device__ __forceinline__ void softmax_role(const Plan& P, Control& C, int cta, int ctas, int half) {
  using Y = Layout<D, PAIR>;
  constexpr int EACH = PAIR ? 2 : 1;  // a half takes every tile, or every other one
  constexpr float SHIFT = std::is_same<T, __half>::value ? 7.0f : 0.0f;
  const int t = threadIdx.x % TILE, warp = t / 32, lane = t % 32;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t tm_s = C.tmem + half * TILE + lanes, tm_o = C.tmem + 2 * TILE + half * D + lanes;
  uint32_t* status = P.L.status;
  Walk<Y::HALVES> walk(C);
  const Segment& s = walk.s;
  uint32_t tile = 0, segment = 0, ends = 0;  // tiles of this half, segments, segments with a tile of this half so far
  bool ok = true;  // uniform over the warp; a warp that has given up still meets the others at barriers
  for (; walk.next(P); ++segment) {
    const int local = (PAIR ? 0 : half * P.half_rows) + t, row = s.row0 + local;
    const bool in_call = t < P.half_rows && row < P.rows;
    const int i = node_of_row(P, row), g = row - i * P.group;
    const int node = P.L.nodes.begin + i;
    const bool live = in_call && node < s.cnt;
    const bool warp_live = __any_sync(FULL, live);
    const int first_masked = s.clear / TILE;  // tiles from here on are not seen whole by every row
    float ref = -INFINITY, sum = 0.0f;

    for (int j = s.first + (PAIR ? half : 0); j < s.last; j += EACH, ++tile) {
      const int base = j * TILE;
      const bool masked = base + TILE > s.clear;
      Seen v;
      auto seen = [&] {
        const int32_t* parent = P.L.nodes.parent + static_cast<int64_t>(s.b) * P.L.nodes.stride;
        return seen_of(P, s, live ? node : -1, base, [&](int n) {
          const int up = C.up[segment % 2][n];
          return up == 0 ? -1 : (up == 255 ? parent[n] : n - up);
        });
      };
      if (!PAIR && masked) {
        // while the scores are made (a segment's first ones say that its parents
        // are there): a tree of 244 rows 36.7 -> 35.4 us, but with the halves
        // taking turns at the tiles 37.0 -> 38.1
        if (j == s.first) ok = ok && warp_wait(&C.s_full[half], tile & 1, C, status);
        v = seen();
      }
      ok = ok && warp_wait(&C.s_full[half], tile & 1, C, status);
      if (warp_live && ok) {
        tmem_fence_after();
        uint32_t x[TILE];
        if (masked) {
          if (PAIR) v = seen();
#pragma unroll 1
          for (int c = 0; c < TILE / 32; ++c) {
            const uint32_t word = live ? v.get(c) : 0xffffffffu;
            if (__all_sync(FULL, word == 0xffffffffu)) continue;
            tmem_ld32(tm_s + c * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((word >> e) & 1)) x[e] = 0xff800000u;
            tmem_st32(tm_s + c * 32, x);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int c = 0; c < TILE / 32; ++c) tmem_ld32(tm_s + c * 32, x + c * 32);
        tmem_wait_ld();
        float top8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) top8[c] = fmaxf(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
#pragma unroll
        for (int c = 16; c < TILE; c += 2)
          top8[c / 2 % 8] = max3(top8[c / 2 % 8], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        const float top = P.scale2 * fmaxf(max3(max3(top8[0], top8[1], top8[2]), top8[3], top8[4]),
                                           max3(top8[5], top8[6], top8[7]));
        const bool grow = live && top > ref + LAZY;
        if (j < s.first + EACH) {
          ref = top;
        } else if (__any_sync(FULL, grow)) {
          const float f = grow ? ex2(ref - top) : 1.0f;
          if (grow) ref = top;
          sum *= f;
#pragma unroll 1
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
        auto weigh = [&](int c) {
          float a, b;
          fma2(F2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), scale2, shift2).get(a, b);
          a = ex2(a);
          b = ex2(b);
          part[c / 2 % 4] = add2(part[c / 2 % 4], F2(a, b));
          x[c / 2] = Pair<T>::pack(a, b);
        };
#pragma unroll
        for (int c = 0; c < EARLY; c += 2) weigh(c);
        tmem_st32(tm_s, x);
        tmem_wait_st();
        tmem_fence_before();
        warp_arrive(&C.w_full[half][0]);
#pragma unroll
        for (int c = EARLY; c < TILE; c += 2) weigh(c);
        tmem_st32(tm_s + EARLY / 2, x + EARLY / 2);
        tmem_wait_st();
        tmem_fence_before();
        float a, b;
        add2(add2(part[0], part[1]), add2(part[2], part[3])).get(a, b);
        sum += a + b;
      } else {
        warp_arrive(&C.w_full[half][0]);
      }
      warp_arrive(&C.w_full[half][1]);
    }

    const bool mine = s.first + (PAIR ? half : 0) < s.last;
    if (mine) ok = ok && warp_wait(&C.o_full[half], ends++ & 1, C, status);
    // PAIR: warp w + 4 hands its rows' statistics to warp w, which puts both
    // outputs together, and goes on when warp w has read them
    const bool both = PAIR && s.last - s.first > 1;
    float f0 = 1.0f, f1 = 0.0f;
    if (both) {
      if (half == 1) {
        C.pair[t] = make_float2(ref, sum);
        tmem_fence_before();
        warps_meet(1 + warp, 64);
        warps_meet(5 + warp, 64);
        tmem_fence_after();
        continue;
      }
      warps_meet(1 + warp, 64);
      const float2 other = C.pair[t];
      const float top = fmaxf(ref, other.x), sub = top == -INFINITY ? 0.0f : top;
      f0 = ex2(ref - sub);
      f1 = ex2(other.x - sub);
      sum = sum * f0 + other.y * f1;
      ref = top;
    } else if (PAIR && half == 1) {
      continue;
    }
    if (!ok || !__any_sync(FULL, in_call)) {
      if (both) warps_meet(5 + warp, 64);
      continue;
    }
    tmem_fence_after();
    const bool whole = s.first == 0 && s.last == s.tiles;
    const Workspace ws = workspace_of(P.L.workspace, P.L.num_sms, P.ws_rows);
    const int64_t part = cta * 2 + (s.first == 0 ? 1 : 0);
    int from = cta, parts = 1;  // of the item: its first CTA, and how many have a part of it
    if (C.pieces) {
      from = cta - C.piece;
      parts = C.pieces;
    } else if (!whole) {
      if (s.first > 0) from = range_of(C.total, s.begin, ctas);
      parts = (s.last == s.tiles ? cta : range_of(C.total, s.begin + s.tiles - 1, ctas)) - from + 1;
    }
    // Ranges: the first CTA puts the parts together if the others are there,
    // with join_rows' operations in their order: the bits do not depend on who
    // does it.
    uint32_t* arrived = ws.arrived + from * 8 + half * 4 + warp;
    bool rest_there = false;
    float top = ref, total = sum;
    if (!whole && !C.pieces && !P.join_inside && s.first == 0 && parts <= JOIN_PARTS) {
      uint32_t n = 0;
      if (lane == 0) n = load_acquire(arrived);
      rest_there = __shfl_sync(FULL, n, 0) + 1 == static_cast<uint32_t>(parts);
      __syncwarp();  // a shuffle orders no memory: the lanes' loads of the parts behind lane 0's acquire
      if (rest_there) {
        float2 ms[JOIN_PARTS - 1];
#pragma unroll
        for (int p = 1; p < JOIN_PARTS; ++p)
          ms[p - 1] = live && p < parts ? __ldcg(&ws.sums[static_cast<int64_t>(from + p) * 2 * P.ws_rows + local])
                                        : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int p = 1; p < JOIN_PARTS; ++p) top = fmaxf(top, ms[p - 1].x);
        const float sub = top == -INFINITY ? 0.0f : top;
        total = sum * ex2(ref - sub);
#pragma unroll
        for (int p = 1; p < JOIN_PARTS; ++p) total = fmaf(ms[p - 1].y, ex2(ms[p - 1].x - sub), total);
      }
    }
    bool finish = whole || rest_there;
    const float top0 = top == -INFINITY ? 0.0f : top, own = rest_there ? ex2(ref - top0) : 1.0f;
    const bool some = live && total != 0.0f;
    const float inv = some ? 1.0f / total : 0.0f;
    T* out = static_cast<T*>(P.L.out.data) + s.b * P.L.out.tree_stride + i * P.L.out.node_stride +
             (static_cast<int64_t>(s.head) * P.group + g) * P.L.out.head_stride;
    float4* partial = ws.out + part * (D / 4) * P.ws_rows + local;
    bool counts, again;  // the row's values count; some row's output is not finite though they do
#pragma unroll 1
    for (;;) {
      Finite finite;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(tm_o + c * 32, o);
        if (both) {
          uint32_t o1[32];
          tmem_ld32(tm_o + D + c * 32, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
        } else {
          tmem_wait_ld();
        }
        if (rest_there && live) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * own);
#pragma unroll 1
          for (int p = 1; p < parts; ++p) {
            const int64_t at = static_cast<int64_t>(from + p) * 2;
            const float4* theirs = ws.out + (at * (D / 4) + c * 8) * P.ws_rows + local;
            const float f = ex2(__ldcg(&ws.sums[at * P.ws_rows + local].x) - top0);
            float4 y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = __ldcg(theirs + q * P.ws_rows);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              o[q * 4] = __float_as_uint(fmaf(y[q].x, f, __uint_as_float(o[q * 4])));
              o[q * 4 + 1] = __float_as_uint(fmaf(y[q].y, f, __uint_as_float(o[q * 4 + 1])));
              o[q * 4 + 2] = __float_as_uint(fmaf(y[q].z, f, __uint_as_float(o[q * 4 + 2])));
              o[q * 4 + 3] = __float_as_uint(fmaf(y[q].w, f, __uint_as_float(o[q * 4 + 3])));
            }
          }
        }
        finite.take(o);
        if (!finish) {
          if (live) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              partial[(c * 8 + q) * P.ws_rows] = make_float4(__uint_as_float(o[q * 4]), __uint_as_float(o[q * 4 + 1]),
                                                             __uint_as_float(o[q * 4 + 2]), __uint_as_float(o[q * 4 + 3]));
          }
        } else if (in_call) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = some ? __uint_as_float(o[q * 8 + e]) * inv : 0.0f;
            *reinterpret_cast<uint4*>(out + c * 32 + q * 8) = pack8<T>(y);
          }
        }
      }
      // no weights, or NaN among them: the row is all zeros or all NaN, whatever the values
      counts = live && (finish ? total != 0.0f && !isnan(total) : !isnan(sum));
      again = __any_sync(FULL, counts && !finite.all());
      if (__builtin_expect(!again || !rest_there, 1)) break;
      rest_there = finish = false;  // parts that are not finite are left to join_rows alone
    }
    if (rest_there && lane == 0) *arrived = 0;
    uint32_t odd = 0;
    for (int x = (max(s.first, first_masked) - first_masked) * (TILE / 32); x < (s.last - first_masked) * (TILE / 32); ++x)
      odd |= C.odd[segment % 3][x];
    if (__builtin_expect(again || odd, 0)) {
      const Segment copy = s;  // the callee takes its address, and s is to stay in registers
      settle<T, D>(P, copy, C.odd[segment % 3], again, counts, node, finish ? out : nullptr, reinterpret_cast<float*>(partial));
    }
    if (!finish && live) ws.sums[part * P.ws_rows + local] = make_float2(ref, sum);
    tmem_fence_before();
    if (both) warps_meet(5 + warp, 64);
    if (finish) continue;
    if (P.join_inside || !C.pieces) {
      // this part is there; the last to say so for its rows puts them together.
      // Lane 0's fences stand between the lanes' stores and its count, and between
      // its count and their loads of the other parts.
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0) {
        __threadfence();
        before = atomicAdd(arrived, 1);
        __threadfence();
      }
      const bool last = __shfl_sync(FULL, before, 0) + 1 == static_cast<uint32_t>(parts);
      __syncwarp();
      if (last) {
        if (lane == 0) *arrived = 0;
        join_rows<T, D>(P, ws, JoinRecord{parts, s.b, s.row0, s.head}, s.cnt, from, local - lane,
                        min(32, P.half_rows - warp * 32), lane, 32);
      }
      __syncwarp();
    } else if (s.first == 0 && local == 0) {
      ws.records[cta] = JoinRecord{parts, s.b, s.row0, s.head};
    }
  }
}

// Where this CTA's range begins: a scan of all items' tiles over all threads.
template <int HALVES>
__device__ __forceinline__ void find_range(const Plan& P, Control& C, int warp, int cta) {
  const int groups = P.L.B * P.row_tiles, per = (groups + THREADS - 1) / THREADS, heads = P.L.kv.n_kv_heads;
  const int x0 = min(groups, static_cast<int>(threadIdx.x) * per), x1 = min(groups, x0 + per);
  int64_t mine = 0;
#pragma unroll 1
  for (int x = x0; x < x1; ++x) mine += group_tiles<HALVES>(P, x);
  mine *= heads;
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(FULL, before, o);
    if (threadIdx.x % 32 >= o) before += up;
  }
  if (threadIdx.x % 32 == 31) C.scan[warp] = before;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += C.scan[w];
    total += C.scan[w];
  }
  before -= mine;
  const int ctas = static_cast<int>(min64(gridDim.x, total));
  const int64_t from = range_start(total, min(cta, ctas), ctas), to = range_start(total, min(cta + 1, ctas), ctas);
  if (threadIdx.x == 0) {
    C.total = total;
    C.count = to - from;
    C.pieces = 0;
  }
  if (from < to && before <= from && from < before + mine) {
    int64_t skip = from - before;
    int x = x0, tiles;
    while (skip >= static_cast<int64_t>(tiles = group_tiles<HALVES>(P, x)) * heads) {
      skip -= static_cast<int64_t>(tiles) * heads;
      ++x;
    }
    Segment& s = C.start;
    s.b = x / P.row_tiles;
    s.rt = x - s.b * P.row_tiles;
    s.head = static_cast<int>(skip / tiles);
    s.first = static_cast<int>(skip - static_cast<int64_t>(s.head) * tiles);
    s.begin = from - s.first;
    set_item<HALVES>(P, s, false);
  }
}

// In tiles of 128 rows (a tile of 256 counts for two): what leaving and joining
// parts costs, and the second segment that a range has.  Estimates: a tile of 256
// rows takes 1.45 us, joining 7 us and a segment's end 5 us of 8 trees' calls.  The
// first weighs against items left whole, the second against ranges.  Pieces and
// ranges, each forced: one token of 4 sequences of 4000 tokens 16.5 and 21.8 us, of
// 16 of 2300 28.2 and 32.6, one tree of 61 nodes over 8192 tokens 34.3 and 55.5,
// 8 over 2300 35.0 and 38.4, 16 over 2300 44.7 and 51.5.
constexpr float JOIN_COST = 6.0f, ENDS_COST = 10.0f;

// Pieces of an item of `tiles` tiles when a piece is to have about 1 / inv.
__device__ __forceinline__ int pieces_of(int tiles, float inv) {
  return max(1, min(tiles, static_cast<int>(ceilf(tiles * inv - 0.001f))));
}

// For no more items than CTAs: the length of equal pieces that costs least, of
// those for which there are CTAs enough, and this CTA's piece.  False: ranges,
// which always have parts to join and begin and end inside items, cost less.
// One lane tries one of 32 lengths, evenly spaced between a range's and the longest
// item's.  Few items of very many tiles lie between two of them, leave CTAs idle
// or go to ranges with more parts than these can join early: 131072 tokens of one
// key head take 66 us, and 44 if pieces are forced; one tree over 65000 tokens of
// one key head 275 and 64, of eight 96.6 and 89.1.
template <int HALVES>
__device__ __forceinline__ bool find_piece(const Plan& P, Control& C, int warp, int cta) {
  const int items = P.L.B * P.row_tiles, heads = P.L.kv.n_kv_heads, lane = threadIdx.x % 32;
  for (int x = threadIdx.x; x < items; x += THREADS) C.tiles[x] = group_tiles<HALVES>(P, x);
  __syncthreads();
  int sum = 0, most = 1;  // 2^31 slots at most in a tree: 2^24 tiles in each of 2^8 items
  float total = 0.0f;
  for (int x = lane; x < items; x += 32) {
    total += static_cast<float>(C.tiles[x]);
    most = max(most, C.tiles[x]);
  }
  total = warp_sum(total) * heads;
  most = __reduce_max_sync(FULL, most);
  constexpr float JOIN = JOIN_COST / HALVES, ENDS = ENDS_COST / HALVES;
  const float fair = __fdividef(total, static_cast<float>(gridDim.x));
  const int least = max(1, static_cast<int>(fair));
  const float inv = __fdividef(1.0f, least + static_cast<float>(max(0, most - least)) * lane * (1.0f / 31.0f));
  float longest = 0.0f;
  bool split = false;
#pragma unroll 4
  for (int x = 0; x < items; ++x) {
    const int n = pieces_of(C.tiles[x], inv);
    sum += n;
    split |= n > 1;
    longest = fmaxf(longest, __fdividef(static_cast<float>(C.tiles[x]), static_cast<float>(n)));
  }
  // the longest length leaves every item whole, so one is always possible
  const float cost = sum * heads <= static_cast<int>(gridDim.x) ? longest + (split ? JOIN : 0.0f) : INFINITY;
  float best = cost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(FULL, best, o));
  if (best > fair + JOIN + ENDS) return false;
  const float chosen = __shfl_sync(FULL, inv, __ffs(__ballot_sync(FULL, cost == best)) - 1);
  if (threadIdx.x == 0) {
    int skip = cta, x = 0, n = 0;
    for (; x < items; ++x) {
      n = pieces_of(C.tiles[x], chosen);
      if (skip < n * heads) break;
      skip -= n * heads;
    }
    C.count = 0;
    C.pieces = n;
    if (x < items) {
      // fewer than 2^8 pieces of at most 2^24 tiles
      const uint32_t tiles = C.tiles[x], head = static_cast<uint32_t>(skip) / n, q = skip - head * n;
      Segment& s = C.start;
      C.piece = q;
      s.b = P.row_tiles == 1 ? x : x / P.row_tiles;
      s.rt = x - s.b * P.row_tiles;
      s.head = head;
      s.first = tiles * q / n;
      s.begin = 0;
      C.count = tiles * (q + 1) / n - s.first;
      set_item<HALVES>(P, s, false);
    }
  }
  return true;
}

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
  if (!P.may_piece || !find_piece<Y::HALVES>(P, C, warp, cta)) find_range<Y::HALVES>(P, C, warp, cta);
  if (threadIdx.x == 0 && P.may_piece) workspace_of(P.L.workspace, P.L.num_sms, P.ws_rows).records[cta].parts = 0;
  if (cta == 0)
    for (int b = threadIdx.x; b < P.L.B; b += THREADS) {
      int len, cnt;
      if (const uint32_t bad = tree_of(P, b, len, cnt)) set_status(P.L.status, bad);
    }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();

  // a softmax thread holds a row of 128 scores in registers: of the 168 each
  // thread starts with, the helpers give some up
  if (warp < HELPERS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    softmax_role<T, D, PAIR>(P, C, cta, static_cast<int>(min64(gridDim.x, C.total)), warp / 4);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
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

// CTA (x, y) of the join: a slice of the elements of the item whose first piece
// was CTA x's.
constexpr int JOIN_THREADS = 256, JOIN_SLICES = 4;

template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) attend_join_kernel(const __grid_constant__ Plan P) {
  grid_dependency_wait();
  grid_dependents_launch();
  const Workspace ws = workspace_of(P.L.workspace, P.L.num_sms, P.ws_rows);
  const JoinRecord rec = ws.records[blockIdx.x];
  if (rec.parts == 0) return;
  int len, cnt;
  tree_of(P, rec.b, len, cnt);
  join_rows<T, D>(P, ws, rec, cnt, blockIdx.x, 0, P.ws_rows, blockIdx.y * JOIN_THREADS + threadIdx.x, JOIN_THREADS * JOIN_SLICES);
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

// Boxes of 64 elements by `box` of a 4-dimensional array of 16-bit elements.
bool tiled_map(CUtensorMap* map, int dtype, const void* base, const cuuint64_t (&dims)[4], const int64_t (&strides)[3],
               int box1, int box2) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  cuuint64_t bytes[3];
  for (int i = 0; i < 3; ++i)  // the stride of a single entry means nothing
    bytes[i] = dims[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(strides[i]) * 2;
  const cuuint32_t boxes[4] = {PANEL, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), 1}, steps[4] = {1, 1, 1, 1};
  return fn(map, dtype == SPEC_TREE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, bytes, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One layer's keys or values, [page][head][token][element]: `box` tokens of
// one head and page.
bool pool_map(CUtensorMap* map, const spec_tree_kv_t& kv, void* base, int layer, int box) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(kv.page_size),
                              static_cast<cuuint64_t>(kv.n_kv_heads), static_cast<cuuint64_t>(kv.n_pages)};
  const int64_t strides[3] = {kv.token_stride, kv.head_stride, kv.page_stride};
  return tiled_map(map, kv.dtype, static_cast<uint16_t*>(base) + layer * kv.layer_stride, dims, strides, box, 1);
}

// Queries, [tree][node][head][element]: one key head's heads of q_box nodes.
bool query_map(CUtensorMap* map, const Plan& P) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(P.L.kv.head_dim), static_cast<cuuint64_t>(P.L.n_q_heads),
                              static_cast<cuuint64_t>(P.L.nodes.count), static_cast<cuuint64_t>(P.L.B)};
  const int64_t strides[3] = {P.L.q.head_stride, P.L.q.node_stride, P.L.q.tree_stride};
  return tiled_map(map, P.L.kv.dtype, P.L.q.data, dims, strides, P.group, P.q_box);
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
  static std::atomic<uint64_t> prepared{0};  // devices that know the kernel's shared memory
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    err = cudaFuncSetAttribute(attend_kernel<T, D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (err != cudaSuccess) return err;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
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
  const Workspace w = workspace_of(nullptr, num_sms, workspace_rows(rows));
  return reinterpret_cast<size_t>(w.out) + static_cast<size_t>(num_sms) * 2 * workspace_rows(rows) * head_dim * 4;
}

cudaError_t launch_attend(const AttendLaunch& L, cudaStream_t stream) {
  Plan P;
  P.L = L;
  P.group = L.n_q_heads / L.kv.n_kv_heads;
  P.rows = L.nodes.count * P.group;
  P.half_rows = TILE / P.group * P.group;
  P.q_box = std::min(TILE / P.group, L.nodes.count);
  P.page_shift = log2_of(L.kv.page_size);
  P.box = L.kv.page_size < TILE ? L.kv.page_size : TILE;
  P.join_inside = P.rows <= JOIN_INSIDE_ROWS;
  // a scale of zero would turn -inf into NaN: weights 2^(1e-30 S) are all one as well
  P.scale2 = fminf(fmaxf(fabsf(L.scale) * 1.4426950408889634f, 1e-30f), 3e38f);
  P.negative = L.scale < 0.0f;
  P.group_inv = P.group == 1 ? 0 : UINT64_MAX / P.group + 1;
  if (L.kv.dtype == SPEC_TREE_BF16)
    return L.kv.head_dim == 128 ? attend_rows<__nv_bfloat16, 128>(P, stream) : attend_rows<__nv_bfloat16, 64>(P, stream);
  return L.kv.head_dim == 128 ? attend_rows<__half, 128>(P, stream) : attend_rows<__half, 64>(P, stream);
}

}  // namespace st
