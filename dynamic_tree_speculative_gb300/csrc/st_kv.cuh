// Device helpers of the paged key-value cache, its appends and its attention.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "st_common.cuh"

namespace st {

// Pairs of float32 that one instruction works on.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit F2(float2 x) : F2(x.x, x.y) {}
  __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return y;
}

__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y.v) : "l"(a.v), "l"(b.v));
  return y;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 y;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y.v) : "l"(a.v), "l"(b.v));
  return y;
}

// Two 16-bit floats of a 32-bit word, low half first.
template <typename T>
struct Pair;

template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ __half2 pair(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <typename T>
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pair<T>::unpack(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Pair<T>::pack(x[0], x[1]), Pair<T>::pack(x[2], x[3]), Pair<T>::pack(x[4], x[5]),
                    Pair<T>::pack(x[6], x[7]));
}

// Element offset, inside one layer, of entry 0 head 0 of slot `slot` of sequence
// b; -1 when the slot has no page in the table or the pool.
__device__ __forceinline__ int64_t kv_slot_offset(const spec_tree_kv_t& kv, int b, int64_t slot, int page_shift) {
  const int64_t idx = slot >> page_shift;
  if (slot < 0 || idx >= kv.max_pages) return -1;
  const int page = kv.page_table[static_cast<int64_t>(b) * kv.table_stride + idx];
  if (page < 0 || page >= kv.n_pages) return -1;
  return page * kv.page_stride + (slot & (kv.page_size - 1)) * kv.token_stride;
}

// Nodes of tree b that exist.
__device__ __forceinline__ int node_count(const spec_tree_nodes_t& nodes, int b) {
  const int total = nodes.begin + nodes.count;
  if (nodes.n_nodes == nullptr) return total;
  const int n = nodes.n_nodes[b];
  return n < 0 ? 0 : (n < total ? n : total);
}

inline int log2_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

}  // namespace st
