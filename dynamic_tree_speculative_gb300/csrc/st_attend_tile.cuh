// Attention of a tree's nodes over a paged key-value cache, many rows at a time:
// tiles of 128 tokens through the tensor cores (tcgen05).  attend.cu, over a cache
// of 16 bits, and attend4.cu, over one of 4, say which they are (CODES) and include this.
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
// Codes.  Keys and values become f16 numbers, and queries too, for any model: with the
// 8 bits of bf16 for keys, values and weights, outputs were 3 times as far from the exact ones as
// their own rounding (and with codes multiplied as they are, scales and zeros applied to each score
// and weight in the softmax, a tree of 64 took 439 us).  Powers of two keep them in
// range: one for a row of queries; for the keys and for the values of each tile, which go
// back in with the scores, the values' into the exponent of the weights; the weights' reference
// so follows scores times values.  (Powers of two for 16 tokens cost 8 times the operations
// beside the weights: a tree of 61 nodes after 4500 tokens, 64 sequences, 287 us instead of 252.)
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
#pragma once

#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "st_attend.cuh"
#include "st_kernels.h"
#include "st_kv.cuh"
#include "st_tensor.cuh"

namespace st {
namespace {

constexpr int PANEL_BYTES = TILE * 128;         // 128 rows of 64 elements
constexpr int MAX_SLOTS = CODES ? 3 : 5;        // of a ring
constexpr int MASKED_TILES = SPEC_TREE_MAX_NODES / TILE + 2;
// Codes: tiles whose scales and zeros are held for the unpacking warps, and whose powers
// of two for the softmax, which is a ring of values behind those.
constexpr int SCALE_SLOTS = CODES ? 6 : 1, POWER_SLOTS = CODES ? SCALE_SLOTS + MAX_SLOTS + 1 : 1;
// Segments whose notes on values are held.  A side warp of values waits for the products
// of the segment before.  One of scales is ahead by what is held of them and by a ring
// of values; a tile's product with the values means that the softmax is done with the
// segments before that tile's.
constexpr int ODD_BUFFERS = CODES ? POWER_SLOTS + 1 : 3;
// Two softmax warpgroups and one of helpers, or two: codes are unpacked by six warps.
constexpr int THREADS = (CODES ? 4 : 3) * TILE;
// A softmax thread holds a row of 128 scores in registers: of those that each thread
// starts with, the helpers give some up.
constexpr int LAUNCH_REGS = CODES ? 128 : 168, SOFTMAX_REGS = CODES ? 200 : 216, HELPER_REGS = CODES ? 56 : 72;
static_assert(2 * SOFTMAX_REGS + (THREADS / TILE - 2) * HELPER_REGS <= THREADS / TILE * LAUNCH_REGS, "registers");
constexpr int HELPERS = 2 * TILE / 32;          // the helpers' first warp
constexpr int COLUMNS = 512;                    // tensor memory: S of both halves, then O of both
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

template <int D, bool PAIR>
struct Layout {
  static constexpr int HALVES = PAIR ? 1 : 2;  // of an item's rows
  static constexpr int PANELS = D / PANEL;
  static constexpr int KV_BYTES = PANELS * PANEL_BYTES;
  static constexpr int Q_BYTES = HALVES * KV_BYTES;
  // tiles that the rings of keys and of values hold: what 7 * 32 KB leave, or 6 beside
  // the rings of codes
  static constexpr int SLOTS = ((CODES ? 6 : 7) * 32768 - Q_BYTES) / KV_BYTES;
  static constexpr int MORE = (SLOTS + 1) / 2 < MAX_SLOTS ? (SLOTS + 1) / 2 : MAX_SLOTS;
  static constexpr int LESS = SLOTS / 2 < MAX_SLOTS ? SLOTS / 2 : MAX_SLOTS;
  static constexpr int KS = CODES ? LESS : MORE, VS = CODES ? MORE : LESS;
};

struct Control : Deal<THREADS / 32> {
  uint64_t k_full[MAX_SLOTS], k_empty[MAX_SLOTS], v_full[MAX_SLOTS], v_empty[MAX_SLOTS], v_clean[MAX_SLOTS];
  uint64_t q_full, q_empty, s_full[2], w_full[2][2], o_full[2], drain;
  uint32_t tmem;
  int abort;
  uint32_t odd[ODD_BUFFERS][MASKED_TILES * (TILE / 32)];  // tokens with a value that is not finite, by segment
  uint8_t up[2][SPEC_TREE_MAX_NODES];           // node minus parent, by segment modulo 2; 0: none, 255: more
  uint2 scales[CODES ? SCALE_SLOTS : 1][CODES ? TILE : 1];  // codes: a token's four numbers
  // codes, by tile: what its products with the keys are to be multiplied by; e and 2^-e, its values being multiplied by
  // the latter; what its keys are
  float4 powers[POWER_SLOTS];
  uint64_t scale_full[SCALE_SLOTS], scale_empty[SCALE_SLOTS];
  uint64_t q_ready;  // codes: queries have been put in order
  union {
    float2 pair[TILE];         // the odd tiles' (reference, sum)
    int tiles[MAX_PIECE_ITEMS];  // setup: tiles of (tree, rows)
  };
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
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value && !CODES;
  constexpr uint32_t ID_S = mma_descriptor(BF, TILE, false), ID_O = mma_descriptor(BF, D, true);
  constexpr int KV16 = Y::KV_BYTES / 16, PANEL16 = PANEL_BYTES / 16;  // descriptors count 16 bytes
  const uint32_t tmem = uniform(C.tmem), q_low = uniform(smem_descriptor_low(q_smem, 0));
  const uint32_t k_low = smem_descriptor_low(k_smem, 0), v_low = smem_descriptor_low(v_smem, PANEL_BYTES);
  uint64_t* queries = CODES ? &C.q_ready : &C.q_full;
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
  // a tile's values (token tile t), cleaned where not every row sees it whole (those made of codes are clean)
  auto values = [&](int t, uint32_t tile) {
    const uint32_t vs = tile % Y::VS;
    if (!warp_wait(&C.v_full[vs], (tile / Y::VS) & 1, C, status)) return false;
    if (!CODES && (t + 1) * TILE > s.clear) {
      if (!warp_wait(&C.v_clean[vs], (clean >> vs) & 1, C, status)) return false;
      clean ^= 1u << vs;
    }
    return true;
  };

  while (walk.next(P)) {
    const int count = s.last - s.first;
    if (!warp_wait(queries, segment & 1, C, status) || !keys(n)) return;
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

// A warp: an item's queries and its nodes' parents into shared memory.
template <int D, bool PAIR>
__device__ __forceinline__ bool ask_queries(const Plan& P, const CUtensorMap* mq, Control& C, uint32_t q_smem, const Segment& s,
                                            uint32_t segment) {
  using Y = Layout<D, PAIR>;
  if (!warp_wait(&C.q_empty, (segment & 1) ^ 1, C, P.L.status)) return false;
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
    for (int x = threadIdx.x % 32; x < s.cnt; x += 32) {
      const int up = parent[x];
      C.up[segment % 2][x] = static_cast<uint8_t>(up < 0 || up >= x ? 0 : min(x - up, 255));
      if (up >= x) set_status(P.L.status, SPEC_TREE_S_NODES);
    }
  }
  warp_arrive(&C.q_full);
  return true;
}

// One warp, ahead of the softmax: queries and parents, and the values of tiles that not every row sees whole: those
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
    ok = ask_queries<D, PAIR>(P, mq, C, q_smem, s, segment);
    if (!ok) break;
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
          if (lane == 0) C.odd[segment % ODD_BUFFERS][(j - first_masked) * (TILE / 32) + part] = word;
        }
        fence_proxy_async_smem();
        warp_arrive(&C.v_clean[slot]);
      }
      warp_arrive(&C.v_empty[slot]);
    }
  }
  if (asked > 0) mbar_wait(&C.q_full, (asked - 1) & 1);  // as load_role: queries in flight land before the CTA ends
}

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

// The accumulator's column of element x (below 32): values made of codes come in
// pairs of elements four apart, which costs nothing to undo here.
__device__ __forceinline__ constexpr int output_column(int x) {
  return CODES ? (x & ~7) + ((x & 3) << 1) + ((x >> 2) & 1) : x;
}

__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The least e with x <= 2^e, from -80 to 126.
__device__ __forceinline__ int power_above(float x) {
  return min(static_cast<int>((__float_as_uint(fmaxf(x, power2(-66))) + 0x007fffffu) >> 23) - 127, 126);
}

// Whether the row's node sees one of the tokens of the segment that `odd` names.
__device__ __noinline__ bool sees_odd(const Plan& P, const Segment& s, const uint32_t* odd, int node) {
  const int first_masked = s.clear / TILE;
  const int32_t* parent = P.L.nodes.parent + static_cast<int64_t>(s.b) * P.L.nodes.stride;
  uint32_t hit = 0;
#pragma unroll 1
  for (int j = max(s.first, first_masked); j < s.last; ++j) {
    const Seen v = seen_of(P, s, node, j * TILE, [&](int n) { return parent[n] < n ? parent[n] : -1; });
    for (int w = 0; w < TILE / 32; ++w) hit |= odd[(j - first_masked) * (TILE / 32) + w] & v.get(w);
  }
  return hit != 0;
}

// 128 threads, one row each: weights, the running reference and sum, and the
// output.
template <typename T, int D, bool PAIR>
__device__ __forceinline__ void softmax_role(const Plan& P, Control& C, uint8_t* q_smem, int cta, int ctas, int half) {
  using Y = Layout<D, PAIR>;
  constexpr int EACH = PAIR ? 2 : 1;  // a half takes every tile, or every other one
  using W = std::conditional_t<CODES, __half, T>;  // weights
  constexpr float SHIFT = std::is_same<W, __half>::value ? 7.0f : 0.0f;
  const int t = threadIdx.x % TILE, warp = t / 32, lane = t % 32;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t tm_s = C.tmem + half * TILE + lanes, tm_o = C.tmem + 2 * TILE + half * D + lanes;
  uint32_t* status = P.L.status;
  Walk<Y::HALVES> walk(C);
  const Segment& s = walk.s;
  uint32_t tile = 0, segment = 0, ends = 0;  // tiles of this half, segments, segments with a tile of this half so far
  uint32_t before = 0;  // tiles of the segments before
  bool ok = true;  // uniform over the warp; a warp that has given up still meets the others at barriers
  for (; walk.next(P); before += s.last - s.first, ++segment) {
    const int local = (PAIR ? 0 : half * P.half_rows) + t, row = s.row0 + local;
    const bool in_call = t < P.half_rows && row < P.rows;
    const int i = node_of_row(P, row), g = row - i * P.group;
    const int node = P.L.nodes.begin + i;
    const bool live = in_call && node < s.cnt;
    const bool warp_live = __any_sync(FULL, live);
    const int first_masked = s.clear / TILE;  // tiles from here on are not seen whole by every row
    float ref = -INFINITY, sum = 0.0f;
    // codes: the row's query as f16 numbers, up to 2^14, in the order in which keys are unpacked
    float factor = 1.0f;
    if (CODES) {
      ok = ok && warp_wait(&C.q_full, segment & 1, C, status);
      if (ok && (!PAIR || half == 0)) {
        uint8_t* own = q_smem + (PAIR ? 0 : half) * Y::KV_BYTES + t * 128;
        float largest = 0.0f;
        auto piece = [&](int c) { return reinterpret_cast<uint4*>(own + c / 8 * PANEL_BYTES + ((c ^ t) % 8) * 16); };
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          float q[8];
          unpack8<T>(*piece(c), q);
#pragma unroll
          for (int e = 0; e < 8; ++e) largest = fmaxf(largest, fabsf(q[e]));
        }
        const int e = power_above(largest);
        const float up = power2(14 - e);
        factor = power2(e - 14);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          float q[8];
          unpack8<T>(*piece(c), q);
          const uint32_t w[4] = {Pair<__half>::pack(q[0] * up, q[4] * up), Pair<__half>::pack(q[1] * up, q[5] * up),
                                 Pair<__half>::pack(q[2] * up, q[6] * up), Pair<__half>::pack(q[3] * up, q[7] * up)};
          *piece(c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (PAIR) C.pair[t].x = factor;
        fence_proxy_async_smem();
      }
      warp_arrive(&C.q_ready);
      if (PAIR && half == 1) {
        ok = ok && warp_wait(&C.q_ready, segment & 1, C, status);
        factor = C.pair[t].x;
      }
    }

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
        float top;
        const float4 power = C.powers[CODES ? (before + j - s.first) % POWER_SLOTS : 0];
        // a zero would make NaN of the -inf of what is not seen
        const float scale = CODES ? fmaxf(power.x * factor, 1e-37f) : P.scale2;
        float top8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) top8[c] = fmaxf(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
#pragma unroll
        for (int c = 16; c < TILE; c += 2)
          top8[c / 2 % 8] = max3(top8[c / 2 % 8], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        top = scale * fmaxf(max3(max3(top8[0], top8[1], top8[2]), top8[3], top8[4]), max3(top8[5], top8[6], top8[7]));
        if (CODES) top += power.y;
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
        const float shift = CODES ? power.y - sub : -sub;
        const F2 scale2(scale, scale), shift2(shift, shift);
        F2 part[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) part[c] = F2(0.0f, 0.0f);
        auto weigh = [&](int c) {
          float a, b;
          fma2(F2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), scale2, shift2).get(a, b);
          a = ex2(a);
          b = ex2(b);
          part[c / 2 % 4] = add2(part[c / 2 % 4], F2(a, b));
          x[c / 2] = Pair<W>::pack(a, b);
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
        sum = CODES ? fmaf(a + b, power.z, sum) : sum + (a + b);
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
    uint32_t odd = 0;  // tokens of the segment, among those that not every row sees, with a value that is not finite
    for (int x = (max(s.first, first_masked) - first_masked) * (TILE / 32); x < (s.last - first_masked) * (TILE / 32); ++x)
      odd |= C.odd[segment % ODD_BUFFERS][x];
    if (CODES && __builtin_expect(odd, 0) && live) {
      const Segment copy = s;
      if (sees_odd(P, copy, C.odd[segment % ODD_BUFFERS], node)) sum = NAN;
    }
    const bool whole = s.first == 0 && s.last == s.tiles;
    const Workspace ws = workspace_of(P);
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
              o[output_column(q * 4)] = __float_as_uint(fmaf(y[q].x, f, __uint_as_float(o[output_column(q * 4)])));
              o[output_column(q * 4 + 1)] = __float_as_uint(fmaf(y[q].y, f, __uint_as_float(o[output_column(q * 4 + 1)])));
              o[output_column(q * 4 + 2)] = __float_as_uint(fmaf(y[q].z, f, __uint_as_float(o[output_column(q * 4 + 2)])));
              o[output_column(q * 4 + 3)] = __float_as_uint(fmaf(y[q].w, f, __uint_as_float(o[output_column(q * 4 + 3)])));
            }
          }
        }
        if (!CODES) finite.take(o);
        if (!finish) {
          if (live) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              partial[(c * 8 + q) * P.ws_rows] = make_float4(__uint_as_float(o[output_column(q * 4)]), __uint_as_float(o[output_column(q * 4 + 1)]),
                                                             __uint_as_float(o[output_column(q * 4 + 2)]), __uint_as_float(o[output_column(q * 4 + 3)]));
          }
        } else if (in_call) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = some ? __uint_as_float(o[output_column(q * 8 + e)]) * inv : 0.0f;
            *reinterpret_cast<uint4*>(out + c * 32 + q * 8) = pack8<T>(y);
          }
        }
      }
      // no weights, or NaN among them: the row is all zeros or all NaN, whatever the values
      counts = live && (finish ? total != 0.0f && !isnan(total) : !isnan(sum));
      again = !CODES && __any_sync(FULL, counts && !finite.all());
      if (__builtin_expect(!again || !rest_there, 1)) break;
      rest_there = finish = false;  // parts that are not finite are left to join_rows alone
    }
    if (rest_there && lane == 0) *arrived = 0;
    if (!CODES && __builtin_expect(again || odd, 0)) {
      const Segment copy = s;  // the callee takes its address, and s is to stay in registers
      settle<T, D>(P, copy, C.odd[segment % ODD_BUFFERS], again, counts, node, finish ? out : nullptr, reinterpret_cast<float*>(partial));
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

// CTA (x, y) of the join: a slice of the elements of the item whose first piece
// was CTA x's.
constexpr int JOIN_THREADS = 256, JOIN_SLICES = 4;

template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS) attend_join_kernel(const __grid_constant__ Plan P) {
  grid_dependency_wait();
  grid_dependents_launch();
  const Workspace ws = workspace_of(P);
  const JoinRecord rec = ws.records[blockIdx.x];
  if (rec.parts == 0) return;
  int len, cnt;
  tree_of(P, rec.b, len, cnt);
  join_rows<T, D>(P, ws, rec, cnt, blockIdx.x, 0, P.ws_rows, blockIdx.y * JOIN_THREADS + threadIdx.x, JOIN_THREADS * JOIN_SLICES);
}

}  // namespace
}  // namespace st
