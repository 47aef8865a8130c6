// What the attention kernels over a paged key-value cache share: how the tiles of
// a call are dealt to the CTAs, which tokens a row sees, and how the parts of an
// item are put together.
#pragma once

#include <math.h>

#include <atomic>
#include <mutex>

#include "st_kernels.h"
#include "st_kv.cuh"
#include "st_tensor.cuh"

namespace st {
namespace {

constexpr int TILE = 128;             // tokens of a tile
constexpr int PANEL = 64;             // 16-bit elements of a 128-byte row
constexpr float LAZY = 8.0f;          // log2 of what a weight may exceed its reference by
constexpr int MAX_PIECE_ITEMS = 256;  // (tree, rows) of calls that may be dealt in pieces
constexpr int JOIN_PARTS = 4;         // parts of an item joined at a time
constexpr int MAX_SPREAD = 2;         // CTAs on an SM

struct Plan {
  AttendLaunch L;
  int group, rows, half_rows, row_tiles, page_shift, box, ws_rows;
  uint64_t group_inv;  // floor(2^64 / group) + 1, 0 for a group of one
  float scale2;        // |scale| log2(e)
  bool may_piece;      // no more items than CTAs
  bool negative;       // scale < 0: the products take -Q
  bool join_inside;    // no join kernel
  int q_box;           // nodes of a copy of queries
  int slots;           // CTAs at most
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

// The counts lie where they lie for every kernel, so that calls of all kinds can
// use one workspace.
__host__ __device__ inline Workspace workspace_of(void* ws, int num_sms, int slots, int ws_rows) {
  Workspace w;
  w.arrived = static_cast<uint32_t*>(ws);
  w.records = reinterpret_cast<JoinRecord*>(w.arrived + num_sms * MAX_SPREAD * 8);
  w.sums = reinterpret_cast<float2*>(w.records + num_sms);
  w.out = reinterpret_cast<float4*>(w.sums + static_cast<size_t>(slots) * 2 * ws_rows);
  return w;
}

__device__ __forceinline__ Workspace workspace_of(const Plan& P) {
  return workspace_of(P.L.workspace, P.L.num_sms, P.slots, P.ws_rows);
}

// A consecutive piece of an item's tiles: what one CTA does at a time.
struct Segment {
  int b, rt, head, row0;   // row0: first row of the item
  int len, cnt;            // committed tokens, nodes that exist
  int first, last, tiles;  // tiles first .. last - 1 of `tiles`
  int end;                 // tokens (slots) the item reads
  int clear;               // slots below this one are seen by every row of the item
  int64_t begin;           // where the item begins among all tiles (ranges)
};

// What a CTA has to do, found by find_piece or find_range.
template <int WARPS>
struct Deal {
  int64_t scan[WARPS];
  int64_t total;      // tiles of the call (ranges)
  int64_t count;      // this CTA's tiles
  int pieces, piece;  // pieces of this CTA's item (0: ranges), and which one this is
  Segment start;      // where this CTA begins
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

// Where range c of `ctas` (below 2^9) begins, and the range that holds tile
// `at`.  64-bit divisions are long: there are seldom tiles enough for them.
__device__ __forceinline__ int64_t range_start(int64_t total, int c, int ctas) {
  if (total < 1 << 23) return static_cast<uint32_t>(total) * c / ctas;
  return total * c / ctas;
}

__device__ __forceinline__ int range_of(int64_t total, int64_t at, int ctas) {
  const int c = total < 1 << 23 ? static_cast<uint32_t>(at) * ctas / static_cast<uint32_t>(total)
                                : static_cast<int>(at * ctas / total);
  return range_start(total, c + 1, ctas) <= at ? c + 1 : c;
}

// The segments of a CTA, one after the other; every role walks them for itself.
template <int HALVES>
struct Walk {
  Segment s;
  int64_t left;
  bool fresh = true;

  template <int WARPS>
  __device__ __forceinline__ explicit Walk(const Deal<WARPS>& C) : s(C.start), left(C.count) {}

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

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One arrival for a whole warp, after what all its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
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

// An item in parts: four elements of a row become the sum of what is not finite
// among them, if there is any; those of CTA slots 0 and 1 are `stride` apart,
// `first` is the first CTA's slot 0.
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

// Where this CTA's range begins: a scan of all items' tiles over all threads.
template <int HALVES, int WARPS>
__device__ __forceinline__ void find_range(const Plan& P, Deal<WARPS>& C, int warp, int cta) {
  constexpr int THREADS = 32 * WARPS;
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
template <int HALVES, int WARPS>
__device__ __forceinline__ bool find_piece(const Plan& P, Deal<WARPS>& C, int* group, int cta) {
  constexpr int THREADS = 32 * WARPS;
  const int items = P.L.B * P.row_tiles, heads = P.L.kv.n_kv_heads, lane = threadIdx.x % 32;
  for (int x = threadIdx.x; x < items; x += THREADS) group[x] = group_tiles<HALVES>(P, x);
  __syncthreads();
  int sum = 0, most = 1;  // 2^30 slots at most in a tree: 2^23 tiles in each of 2^8 items
  float total = 0.0f;
  for (int x = lane; x < items; x += 32) {
    total += static_cast<float>(group[x]);
    most = max(most, group[x]);
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
    const int n = pieces_of(group[x], inv);
    sum += n;
    split |= n > 1;
    longest = fmaxf(longest, __fdividef(static_cast<float>(group[x]), static_cast<float>(n)));
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
      n = pieces_of(group[x], chosen);
      if (skip < n * heads) break;
      skip -= n * heads;
    }
    C.count = 0;
    C.pieces = n;
    if (x < items) {
      // fewer than 2^9 pieces of at most 2^23 tiles
      const uint32_t tiles = group[x], head = static_cast<uint32_t>(skip) / n, q = skip - head * n;
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

// -------------------------------------------------------------------- host ---

// What all kernels take from a call; the rest is theirs.
inline Plan plan_of(const AttendLaunch& L) {
  Plan P = {};
  P.L = L;
  P.slots = L.num_sms;
  P.group = L.n_q_heads / L.kv.n_kv_heads;
  P.rows = L.nodes.count * P.group;
  P.half_rows = TILE / P.group * P.group;
  P.page_shift = log2_of(L.kv.page_size);
  // a scale of zero would turn -inf into NaN: weights 2^(1e-30 S) are all one as well
  P.scale2 = fminf(fmaxf(fabsf(L.scale) * 1.4426950408889634f, 1e-30f), 3e38f);
  P.negative = L.scale < 0.0f;
  P.group_inv = P.group == 1 ? 0 : UINT64_MAX / P.group + 1;
  return P;
}

// Tells the current device, once, how much shared memory the kernel takes, and
// looks whether it has as many registers a thread as it was written for.
template <auto KERNEL>
cudaError_t prepare_kernel(int bytes, int registers) {
  static std::atomic<uint64_t> prepared{0};
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (!(prepared.load(std::memory_order_relaxed) & bit)) {
    cudaFuncAttributes has;
    if ((err = cudaFuncGetAttributes(&has, KERNEL)) != cudaSuccess) return err;
    if (has.numRegs < registers) return cudaErrorLaunchOutOfResources;
    err = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    prepared.fetch_or(bit, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
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

// Boxes of a 4-dimensional array whose elements have `size` bytes; strides in elements.
struct Boxes {
  cuuint32_t n[4];
};

inline bool tiled_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, const cuuint64_t (&dims)[4],
               const int64_t (&strides)[3], const Boxes& boxes, CUtensorMapSwizzle swizzle) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  cuuint64_t bytes[3];
  for (int i = 0; i < 3; ++i)  // the stride of a single entry means nothing
    bytes[i] = dims[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(strides[i]) * size;
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(map, type, 4, const_cast<void*>(base), dims, bytes, boxes.n, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline CUtensorMapDataType type_of(int dtype) {
  return dtype == SPEC_TREE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

[[maybe_unused]] // Queries, [tree][node][head][element]: one key head's heads of q_box nodes.
inline bool query_map(CUtensorMap* map, const Plan& P) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(P.L.kv.head_dim), static_cast<cuuint64_t>(P.L.n_q_heads),
                              static_cast<cuuint64_t>(P.L.nodes.count), static_cast<cuuint64_t>(P.L.B)};
  const int64_t strides[3] = {P.L.q.head_stride, P.L.q.node_stride, P.L.q.tree_stride};
  return tiled_map(map, type_of(P.L.kv.dtype), 2, P.L.q.data, dims, strides,
                   {PANEL, static_cast<cuuint32_t>(P.group), static_cast<cuuint32_t>(P.q_box), 1}, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace
}  // namespace st
