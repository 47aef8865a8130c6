// Host side of the key-value cache entry points (include/spec_tree.h):
// argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spec_tree.h"
#include "st_kernels.h"

namespace {

constexpr int MAX_CHAIN = 1 << 20;
constexpr int MAX_HEADS = 1 << 14;
constexpr int MAX_TREES = 65535;
constexpr int64_t MAX_SLOTS = 1ll << 30;  // of a sequence
constexpr int MAX_GROUP = 128;            // query heads of a key head
constexpr int64_t MAX_STRIDE = 1ll << 38;  // elements

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

int check_kv(int B, const spec_tree_kv_t* kv, int layer) {
  if (kv == nullptr || B < 0 || B > MAX_TREES) return SPEC_TREE_E_PARAM;
  if (kv->dtype != SPEC_TREE_BF16 && kv->dtype != SPEC_TREE_F16) return SPEC_TREE_E_LAYOUT;
  if (kv->k == nullptr || kv->v == nullptr || kv->page_table == nullptr || kv->seq_len == nullptr)
    return SPEC_TREE_E_PARAM;
  if (kv->n_layers < 1 || layer < 0 || layer >= kv->n_layers || kv->n_pages < 1 || kv->n_kv_heads < 1 ||
      kv->n_kv_heads > MAX_HEADS || kv->max_pages < 1 || kv->table_stride < kv->max_pages)
    return SPEC_TREE_E_PARAM;
  if (kv->head_dim != 64 && kv->head_dim != 128) return SPEC_TREE_E_PARAM;
  if (kv->page_size < 8 || kv->page_size > 65536 || (kv->page_size & (kv->page_size - 1)) != 0)
    return SPEC_TREE_E_PARAM;
  if (static_cast<int64_t>(kv->max_pages) * kv->page_size > MAX_SLOTS) return SPEC_TREE_E_PARAM;
  if (!aligned16(kv->k) || !aligned16(kv->v)) return SPEC_TREE_E_LAYOUT;
  const int64_t st[4] = {kv->layer_stride, kv->page_stride, kv->token_stride, kv->head_stride};
  for (int64_t x : st)
    if (x < 0 || x % 8 != 0 || x >= MAX_STRIDE) return SPEC_TREE_E_LAYOUT;
  return SPEC_TREE_OK;
}

int check_nodes(const spec_tree_nodes_t* n, bool need_depth) {
  if (n == nullptr || n->begin < 0 || n->count < 1) return SPEC_TREE_E_PARAM;
  const int64_t end = static_cast<int64_t>(n->begin) + n->count;
  if (n->parent == nullptr) return n->depth == nullptr && end <= MAX_CHAIN ? SPEC_TREE_OK : SPEC_TREE_E_PARAM;
  if (need_depth && n->depth == nullptr) return SPEC_TREE_E_PARAM;
  return end <= n->stride && end <= SPEC_TREE_MAX_NODES ? SPEC_TREE_OK : SPEC_TREE_E_PARAM;
}

int check_heads(const spec_tree_heads_t* h) {
  if (h == nullptr || h->data == nullptr) return SPEC_TREE_E_PARAM;
  if (!aligned16(h->data)) return SPEC_TREE_E_LAYOUT;
  const int64_t st[3] = {h->tree_stride, h->node_stride, h->head_stride};
  for (int64_t x : st)
    if (x < 0 || x % 8 != 0 || x >= MAX_STRIDE) return SPEC_TREE_E_LAYOUT;
  return SPEC_TREE_OK;
}

int check_kv4(int B, const spec_tree_kv4_t* kv, int layer) {
  if (kv == nullptr) return SPEC_TREE_E_PARAM;
  const int rc = check_kv(B, &kv->kv, layer);
  if (rc) return rc;
  if (kv->scale == nullptr) return SPEC_TREE_E_PARAM;
  const int64_t codes[4] = {kv->kv.layer_stride, kv->kv.page_stride, kv->kv.token_stride, kv->kv.head_stride};
  for (int64_t x : codes)
    if (x % 32 != 0) return SPEC_TREE_E_LAYOUT;  // 16 bytes
  const int64_t scales[3] = {kv->scale_layer_stride, kv->scale_page_stride, kv->scale_head_stride};
  for (int64_t x : scales)
    if (x < 0 || x % 8 != 0 || x >= MAX_STRIDE) return SPEC_TREE_E_LAYOUT;
  return aligned16(kv->scale) ? SPEC_TREE_OK : SPEC_TREE_E_LAYOUT;
}

st::KvScale scales_of(const spec_tree_kv4_t& kv) {
  return st::KvScale{kv.scale, kv.scale_layer_stride, kv.scale_page_stride, kv.scale_head_stride};
}

int check_pages(int B, const spec_tree_pages_t* p) {
  if (p == nullptr || B < 0 || B > MAX_TREES || p->page_table == nullptr || p->held == nullptr || p->free_pages == nullptr ||
      p->n_free == nullptr || p->scratch == nullptr)
    return SPEC_TREE_E_PARAM;
  if (p->n_pages < 1 || p->max_pages < 1 || p->table_stride < p->max_pages || p->page_size < 8 || p->page_size > 65536 ||
      (p->page_size & (p->page_size - 1)) != 0 || static_cast<int64_t>(p->max_pages) * p->page_size > MAX_SLOTS)
    return SPEC_TREE_E_PARAM;
  return SPEC_TREE_OK;
}

cudaStream_t as_stream(spec_tree_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

int of(cudaError_t err) { return err == cudaSuccess ? SPEC_TREE_OK : SPEC_TREE_E_CUDA; }

// What the entry points of both kinds of cache share, behind their own checks of it.
int append(int B, const spec_tree_kv_t* kv, const st::KvScale& scales, int layer, const spec_tree_nodes_t* nodes,
           int n_q_heads, const spec_tree_heads_t* q, const spec_tree_heads_t* k, const spec_tree_heads_t* v,
           const spec_tree_heads_t* q_out, const float* rope, int rope_rows, int rot_dim, int interleaved,
           const void* q_weight, const void* k_weight, float eps, uint32_t* status, spec_tree_stream_t stream) {
  int rc;
  if ((rc = check_nodes(nodes, true))) return rc;
  if (n_q_heads < 1 || n_q_heads > MAX_HEADS ||
      static_cast<int64_t>(B) * nodes->count * (n_q_heads + 2 * kv->n_kv_heads) > INT32_MAX)
    return SPEC_TREE_E_PARAM;
  const spec_tree_heads_t* heads[4] = {q, k, v, q_out};
  for (const spec_tree_heads_t* h : heads)
    if ((rc = check_heads(h))) return rc;
  if (rot_dim < 0 || rot_dim > kv->head_dim || rot_dim % 16 != 0) return SPEC_TREE_E_PARAM;
  if ((rope == nullptr) != (rot_dim == 0) || (rope != nullptr && rope_rows < 1)) return SPEC_TREE_E_PARAM;
  if (!(eps >= 0.0f) || !isfinite(eps)) return SPEC_TREE_E_PARAM;
  if (!aligned16(rope) || !aligned16(q_weight) || !aligned16(k_weight)) return SPEC_TREE_E_LAYOUT;
  if (B == 0) return SPEC_TREE_OK;
  st::AppendLaunch L;
  L.B = B;
  L.layer = layer;
  L.n_q_heads = n_q_heads;
  L.kv = *kv;
  L.nodes = *nodes;
  L.q = *q;
  L.k = *k;
  L.v = *v;
  L.q_out = *q_out;
  L.rope = rope;
  L.rope_rows = rope_rows;
  L.rot_dim = rot_dim;
  L.interleaved = interleaved != 0;
  L.q_weight = q_weight;
  L.k_weight = k_weight;
  L.eps = eps;
  L.status = status;
  L.scales = scales;
  L.num_sms = st::num_sms_of_current_device();
  if (L.num_sms <= 0) return SPEC_TREE_E_CUDA;
  return of(st::launch_kv_append(L, as_stream(stream)));
}

int attend(int B, const spec_tree_kv_t* kv, const st::KvScale& scales, int layer, const spec_tree_nodes_t* nodes,
           int n_q_heads, const spec_tree_heads_t* q, const spec_tree_heads_t* out, float scale, void* workspace,
           size_t workspace_bytes, uint32_t* status, spec_tree_stream_t stream) {
  int rc;
  if ((rc = check_nodes(nodes, false))) return rc;
  if (n_q_heads < kv->n_kv_heads || n_q_heads > MAX_HEADS || n_q_heads % kv->n_kv_heads != 0 ||
      n_q_heads / kv->n_kv_heads > MAX_GROUP || static_cast<int64_t>(B) * nodes->count * n_q_heads > (1 << 30))
    return SPEC_TREE_E_PARAM;
  if ((rc = check_heads(q)) || (rc = check_heads(out))) return rc;
  if (!isfinite(scale) || workspace == nullptr || q->data == out->data) return SPEC_TREE_E_PARAM;
  if (!aligned16(workspace)) return SPEC_TREE_E_LAYOUT;
  if (B == 0) return SPEC_TREE_OK;
  st::AttendLaunch L;
  L.num_sms = st::num_sms_of_current_device();
  if (L.num_sms <= 0) return SPEC_TREE_E_CUDA;
  const int64_t rows = static_cast<int64_t>(nodes->count) * (n_q_heads / kv->n_kv_heads);
  if (workspace_bytes < st::attend_workspace_bytes(L.num_sms, rows, kv->head_dim)) return SPEC_TREE_E_PARAM;
  L.B = B;
  L.layer = layer;
  L.n_q_heads = n_q_heads;
  L.kv = *kv;
  L.nodes = *nodes;
  L.q = *q;
  L.out = *out;
  L.scale = scale;
  L.workspace = workspace;
  L.status = status;
  L.scales = scales;
  return of(scales.data ? st::launch_kv4_attend(L, as_stream(stream)) : st::launch_attend(L, as_stream(stream)));
}

int commit(int B, const spec_tree_kv_t* kv, const st::KvScale& scales, const int32_t* accept_len, const int32_t* out_node,
           int path_stride, int32_t* new_len, uint32_t* status, spec_tree_stream_t stream) {
  if (accept_len == nullptr || out_node == nullptr || new_len == nullptr || new_len == kv->seq_len ||
      path_stride < 1 || path_stride > 256)
    return SPEC_TREE_E_PARAM;
  if (B == 0) return SPEC_TREE_OK;
  st::CommitLaunch L;
  L.B = B;
  L.kv = *kv;
  L.accept_len = accept_len;
  L.out_node = out_node;
  L.path_stride = path_stride;
  L.new_len = new_len;
  L.status = status;
  L.scales = scales;
  return of(scales.data ? st::launch_kv4_commit(L, as_stream(stream)) : st::launch_kv_commit(L, as_stream(stream)));
}

}  // namespace

extern "C" {

int spec_tree_kv_append(int B, const spec_tree_kv_t* kv, int layer, const spec_tree_nodes_t* nodes, int n_q_heads,
                        const spec_tree_heads_t* q, const spec_tree_heads_t* k, const spec_tree_heads_t* v,
                        const spec_tree_heads_t* q_out, const float* rope, int rope_rows, int rot_dim,
                        int interleaved, const void* q_weight, const void* k_weight, float eps, uint32_t* status,
                        spec_tree_stream_t stream) {
  const int rc = check_kv(B, kv, layer);
  return rc ? rc : append(B, kv, st::KvScale(), layer, nodes, n_q_heads, q, k, v, q_out, rope, rope_rows, rot_dim,
                          interleaved, q_weight, k_weight, eps, status, stream);
}

int spec_tree_kv4_append(int B, const spec_tree_kv4_t* kv, int layer, const spec_tree_nodes_t* nodes, int n_q_heads,
                         const spec_tree_heads_t* q, const spec_tree_heads_t* k, const spec_tree_heads_t* v,
                         const spec_tree_heads_t* q_out, const float* rope, int rope_rows, int rot_dim,
                         int interleaved, const void* q_weight, const void* k_weight, float eps, uint32_t* status,
                         spec_tree_stream_t stream) {
  const int rc = check_kv4(B, kv, layer);
  return rc ? rc : append(B, &kv->kv, scales_of(*kv), layer, nodes, n_q_heads, q, k, v, q_out, rope, rope_rows, rot_dim,
                          interleaved, q_weight, k_weight, eps, status, stream);
}

size_t spec_tree_attend_workspace_bytes(int B, int count, int n_q_heads, int n_kv_heads, int head_dim) {
  if (B < 1 || count < 1 || count > MAX_CHAIN || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads > MAX_HEADS ||
      n_q_heads % n_kv_heads != 0 || n_q_heads / n_kv_heads > MAX_GROUP || (head_dim != 64 && head_dim != 128))
    return 0;
  const int sms = st::num_sms_of_current_device();
  return sms <= 0 ? 0 : st::attend_workspace_bytes(sms, static_cast<int64_t>(count) * (n_q_heads / n_kv_heads), head_dim);
}

int spec_tree_attend(int B, const spec_tree_kv_t* kv, int layer, const spec_tree_nodes_t* nodes, int n_q_heads,
                     const spec_tree_heads_t* q, const spec_tree_heads_t* out, float scale, void* workspace,
                     size_t workspace_bytes, uint32_t* status, spec_tree_stream_t stream) {
  const int rc = check_kv(B, kv, layer);
  return rc ? rc : attend(B, kv, st::KvScale(), layer, nodes, n_q_heads, q, out, scale, workspace, workspace_bytes,
                          status, stream);
}

int spec_tree_kv4_attend(int B, const spec_tree_kv4_t* kv, int layer, const spec_tree_nodes_t* nodes, int n_q_heads,
                         const spec_tree_heads_t* q, const spec_tree_heads_t* out, float scale, void* workspace,
                         size_t workspace_bytes, uint32_t* status, spec_tree_stream_t stream) {
  const int rc = check_kv4(B, kv, layer);
  return rc ? rc : attend(B, &kv->kv, scales_of(*kv), layer, nodes, n_q_heads, q, out, scale, workspace, workspace_bytes,
                          status, stream);
}

int spec_tree_kv_commit(int B, const spec_tree_kv_t* kv, const int32_t* accept_len, const int32_t* out_node,
                        int path_stride, int32_t* new_len, uint32_t* status, spec_tree_stream_t stream) {
  const int rc = check_kv(B, kv, 0);
  return rc ? rc : commit(B, kv, st::KvScale(), accept_len, out_node, path_stride, new_len, status, stream);
}

int spec_tree_kv4_commit(int B, const spec_tree_kv4_t* kv, const int32_t* accept_len, const int32_t* out_node,
                         int path_stride, int32_t* new_len, uint32_t* status, spec_tree_stream_t stream) {
  const int rc = check_kv4(B, kv, 0);
  return rc ? rc : commit(B, &kv->kv, scales_of(*kv), accept_len, out_node, path_stride, new_len, status, stream);
}

int spec_tree_kv4_read(int B, const spec_tree_kv4_t* kv, int layer, const int32_t* first, const int32_t* counts, int count,
                       const spec_tree_heads_t* k, const spec_tree_heads_t* v, uint32_t* status, spec_tree_stream_t stream) {
  if (kv == nullptr) return SPEC_TREE_E_PARAM;
  spec_tree_kv4_t with = *kv;
  if (with.kv.seq_len == nullptr) with.kv.seq_len = with.kv.page_table;  // not read
  int rc = check_kv4(B, &with, layer);
  if (rc) return rc;
  if (count < 1 || count > MAX_CHAIN || static_cast<int64_t>(B) * count * kv->kv.n_kv_heads > (1 << 30))
    return SPEC_TREE_E_PARAM;
  if ((rc = check_heads(k)) || (rc = check_heads(v))) return rc;
  if (k->data == v->data) return SPEC_TREE_E_PARAM;
  if (B == 0) return SPEC_TREE_OK;
  st::ReadLaunch L;
  L.B = B;
  L.layer = layer;
  L.count = count;
  L.kv = with.kv;
  L.scales = scales_of(*kv);
  L.first = first;
  L.counts = counts;
  L.k = *k;
  L.v = *v;
  L.status = status;
  return of(st::launch_kv4_read(L, as_stream(stream)));
}

int spec_tree_kv_reserve(int B, const spec_tree_pages_t* pages, const int32_t* seq_len, const int32_t* n_nodes, int count,
                         int64_t* slots, uint32_t* status, spec_tree_stream_t stream) {
  const int rc = check_pages(B, pages);
  if (rc) return rc;
  if (seq_len == nullptr || count < 1 || count > MAX_CHAIN) return SPEC_TREE_E_PARAM;
  if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return SPEC_TREE_E_LAYOUT;
  if (B == 0) return SPEC_TREE_OK;
  return of(st::launch_kv_reserve(st::ReserveLaunch{B, count, *pages, seq_len, n_nodes, slots, status}, as_stream(stream)));
}

int spec_tree_kv_release(int B, const spec_tree_pages_t* pages, const int32_t* keep, uint32_t* status,
                         spec_tree_stream_t stream) {
  const int rc = check_pages(B, pages);
  if (rc) return rc;
  if (keep == nullptr) return SPEC_TREE_E_PARAM;
  if (B == 0) return SPEC_TREE_OK;
  return of(st::launch_kv_release(st::ReleaseLaunch{B, *pages, keep, status}, as_stream(stream)));
}

}  // extern "C"
