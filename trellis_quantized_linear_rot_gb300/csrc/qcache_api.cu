// C ABI of the operators declared in tf_qcache.h: argument checks, then a
// launch on the caller's stream.
#include <cmath>

#include "checks.h"
#include "qcache.h"

using namespace tfx;

namespace {

bool head_dim_served(int d) { return d == 64 || d == 128 || d == 256; }

// Rows of one call that moves rows: their number is a 31-bit one.
bool too_many(int64_t batch, int64_t tokens, int64_t heads) {
  return static_cast<double>(batch) * static_cast<double>(tokens) * static_cast<double>(heads) > 2147483647.0;
}

// The checks of a cache that need no device. nodes: of a tree, or 0.
tf_status check_cache(const tf_kvq_cache* c, int nodes) {
  if (!c) return TF_ERR_NULL;
  if (c->batch < 0 || nodes < 0 || nodes > TF_MAX_NODES || c->layers < 1 || c->pages < 1 || c->page_size < 1 ||
      c->kv_heads < 1 || !head_dim_served(c->head_dim) || c->table_width < 1)
    return TF_ERR_SHAPE;
  if (c->batch > 65535 || c->layers > 65535 || c->kv_heads > 65535 ||
      static_cast<int64_t>(c->table_width) * c->page_size > INT32_MAX - 2 * TF_MAX_NODES)
    return TF_ERR_SHAPE;
  if (c->stride_layer < 0 || c->stride_page < 0 || c->stride_token < 0 || c->stride_head < 0 || c->scale_layer < 0 ||
      c->scale_page < 0 || c->scale_token < 0 || c->scale_head < 0 || c->stride_table < 0)
    return TF_ERR_SHAPE;
  if (c->bits != 4 && c->bits != 8) return TF_ERR_BITS;
  return TF_OK;
}

tf_status check_cache_pointers(const tf_kvq_cache* c) {
  if (!c->k || !c->v || !c->scales || !c->page_table || !c->lengths) return TF_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->scales, 4) || !aligned(c->page_table, 4) ||
      !aligned(c->lengths, 4) || ((c->stride_layer | c->stride_page | c->stride_token | c->stride_head) & 15) ||
      ((c->scale_layer | c->scale_page | c->scale_token | c->scale_head) & 1))
    return TF_ERR_ALIGN;
  return TF_OK;
}

tf_status check_cache_device(const tf_kvq_cache* c, int device) {
  return check_pointers_on_device(device, {c->k, c->v, c->scales, c->page_table, c->lengths});
}

QView view_of(const tf_kvq_cache* c, int* err) {
  QView v;
  v.c.stride_layer = c->stride_layer;
  v.c.stride_page = c->stride_page;
  v.c.stride_token = c->stride_token;
  v.c.stride_head = c->stride_head;
  v.c.page_table = c->page_table;
  v.c.lengths = c->lengths;
  v.c.stride_table = c->stride_table;
  v.c.layers = c->layers;
  v.c.pages = c->pages;
  v.c.page_size = c->page_size;
  v.c.kv_heads = c->kv_heads;
  v.c.head_dim = c->head_dim;
  v.c.batch = c->batch;
  v.c.table_width = c->table_width;
  v.c.by_page = FastDiv(static_cast<uint32_t>(c->page_size));
  v.c.err = err;
  v.scale_layer = c->scale_layer / 2;
  v.scale_page = c->scale_page / 2;
  v.scale_token = c->scale_token / 2;
  v.scale_head = c->scale_head / 2;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.scales = static_cast<uint32_t*>(c->scales);
  v.bits = c->bits;
  return v;
}

bool negative(const tf_head_rows& r) {
  return r.x_seq < 0 || r.x_node < 0 || r.x_head < 0 || r.y_seq < 0 || r.y_node < 0 || r.y_head < 0;
}
bool misaligned(const tf_head_rows& r, int weight_dtype) {
  return !aligned(r.x, 16) || !aligned(r.y, 16) || !aligned(r.weight, weight_dtype == TF_F32 ? 4 : 2) ||
         !eights(r.x_seq, r.x_node, r.x_head) || !eights(r.y_seq, r.y_node, r.y_head);
}

}  // namespace

extern "C" {

tf_status tf_qk_norm_rope(const tf_head_rows* queries, const tf_head_rows* keys, int dtype, int weight_dtype,
                          const int32_t* positions, int64_t stride_positions, const double* inv_freq, int rotary,
                          double eps, int flags, int batch, int nodes, int head_dim, void* stream) {
  if (!queries) return TF_ERR_NULL;
  const tf_head_rows& q = *queries;
  const tf_head_rows none = {};
  const tf_head_rows& k = keys ? *keys : none;
  if (batch < 0 || nodes < 0 || q.heads < 1 || (keys && k.heads < 1) || q.heads > 65535 || k.heads > 65535 ||
      !head_dim_served(head_dim) || rotary < 0 || rotary > head_dim || rotary % 16 || stride_positions < 0 ||
      negative(q) || negative(k) || !(eps >= 0.0) || !(eps <= std::numeric_limits<float>::max()) ||
      (flags & ~(TF_QK_NO_NORM | TF_QK_INTERLEAVED | TF_QK_HADAMARD)) || too_many(batch, nodes, q.heads + k.heads))
    return TF_ERR_SHAPE;
  if ((dtype != TF_F16 && dtype != TF_BF16) ||
      (weight_dtype != TF_F16 && weight_dtype != TF_F32 && weight_dtype != TF_BF16))
    return TF_ERR_DTYPE;
  if (batch == 0 || nodes == 0) return TF_OK;
  if (!q.x || !q.y || (keys && (!k.x || !k.y)) || !positions || (rotary && !inv_freq)) return TF_ERR_NULL;
  if (misaligned(q, weight_dtype) || misaligned(k, weight_dtype) || !aligned(positions, 4) ||
      (rotary && !aligned(inv_freq, 8)))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  tf_status s = current_device_state(&device, &sms, &err);
  if (s == TF_OK) s = check_pointers_on_device(device, {q.x, q.y, positions});
  if (s == TF_OK && keys) s = check_pointers_on_device(device, {k.x, k.y});
  if (s == TF_OK && rotary) s = check_pointers_on_device(device, {inv_freq});
  if (s == TF_OK && q.weight) s = check_pointers_on_device(device, {q.weight});
  if (s == TF_OK && k.weight) s = check_pointers_on_device(device, {k.weight});
  if (s != TF_OK) return s;
  NormRopeArgs a;
  a.q = q;
  a.k = k;
  a.positions = positions;
  a.stride_positions = stride_positions;
  a.inv_freq = inv_freq;
  a.rotary = rotary;
  a.flags = flags;
  a.eps = static_cast<float>(eps);
  a.batch = batch;
  a.nodes = nodes;
  a.num_sms = sms;
  return launched(launch_qk_norm_rope(a, dtype, weight_dtype, head_dim, static_cast<cudaStream_t>(stream)),
                  "norm and rotation launch");
}

tf_status tf_kvq_write(const tf_kvq_cache* cache, const void* k_new, int64_t k_stride_seq, int64_t k_stride_node,
                       int64_t k_stride_head, const void* v_new, int64_t v_stride_seq, int64_t v_stride_node,
                       int64_t v_stride_head, int dtype, const int32_t* counts, int nodes, void* stream) {
  tf_status s = check_cache(cache, 0);
  if (s != TF_OK) return s;
  if (cache->layers != 1 || nodes < 0 || k_stride_seq < 0 || k_stride_node < 0 || k_stride_head < 0 ||
      v_stride_seq < 0 || v_stride_node < 0 || v_stride_head < 0 || too_many(cache->batch, nodes, cache->kv_heads))
    return TF_ERR_SHAPE;
  if (dtype != TF_F16 && dtype != TF_BF16) return TF_ERR_DTYPE;
  if (cache->batch == 0 || nodes == 0) return TF_OK;
  s = check_cache_pointers(cache);
  if (s == TF_ERR_NULL || !k_new || !v_new) return TF_ERR_NULL;
  if (s != TF_OK || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(counts, 4) ||
      !eights(k_stride_seq, k_stride_node, k_stride_head) || !eights(v_stride_seq, v_stride_node, v_stride_head))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  s = current_device_state(&device, &sms, &err);
  if (s == TF_OK) s = check_cache_device(cache, device);
  if (s == TF_OK) s = check_pointers_on_device(device, {k_new, v_new});
  if (s == TF_OK && counts) s = check_pointers_on_device(device, {counts});
  if (s != TF_OK) return s;
  const RowsIn k = {k_new, k_stride_seq, k_stride_node, k_stride_head};
  const RowsIn v = {v_new, v_stride_seq, v_stride_node, v_stride_head};
  return launched(launch_kvq_write(view_of(cache, err), k, v, dtype, counts, nodes, static_cast<cudaStream_t>(stream)),
                  "quantised cache write launch");
}

tf_status tf_kvq_read(const tf_kvq_cache* cache, const int32_t* starts, void* k_out, void* v_out, int dtype,
                      int64_t stride_seq, int64_t stride_slot, int64_t stride_head, int slots, void* stream) {
  tf_status s = check_cache(cache, 0);
  if (s != TF_OK) return s;
  if (cache->layers != 1 || slots < 0 || stride_seq < 0 || stride_slot < 0 || stride_head < 0 ||
      too_many(cache->batch, slots, cache->kv_heads))
    return TF_ERR_SHAPE;
  if (dtype != TF_F16 && dtype != TF_BF16) return TF_ERR_DTYPE;
  if (cache->batch == 0 || slots == 0) return TF_OK;
  s = check_cache_pointers(cache);
  if (s == TF_ERR_NULL || !k_out || !v_out) return TF_ERR_NULL;
  if (s != TF_OK || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(starts, 4) ||
      !eights(stride_seq, stride_slot, stride_head))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  s = current_device_state(&device, &sms, &err);
  if (s == TF_OK) s = check_cache_device(cache, device);
  if (s == TF_OK) s = check_pointers_on_device(device, {k_out, v_out});
  if (s == TF_OK && starts) s = check_pointers_on_device(device, {starts});
  if (s != TF_OK) return s;
  return launched(launch_kvq_read(view_of(cache, err), starts, k_out, v_out, dtype, stride_seq, stride_slot,
                                  stride_head, slots, static_cast<cudaStream_t>(stream)),
                  "quantised cache read launch");
}

size_t tf_kvq_attention_workspace_bytes(int batch, int nodes, int heads, int kv_heads, int head_dim) {
  if (batch < 0 || batch > 65535 || nodes < 0 || nodes > TF_MAX_NODES || heads < 1 || kv_heads < 1 ||
      heads % kv_heads || !head_dim_served(head_dim))
    return 0;
  int device, sms, *err;
  if (current_device_state(&device, &sms, &err) != TF_OK) return 0;
  return kvq_attend_workspace(nodes, heads, kv_heads, head_dim, sms).bytes;
}

tf_status tf_kvq_attention(const tf_kvq_cache* cache, const void* q, int dtype, int64_t q_stride_seq,
                           int64_t q_stride_node, int64_t q_stride_head, const int32_t* parents,
                           int64_t stride_parents, void* out, float* lse, int nodes, int heads, double scale,
                           void* workspace, size_t workspace_bytes, void* stream) {
  tf_status s = check_cache(cache, nodes);
  if (s != TF_OK) return s;
  if (cache->layers != 1 || heads < 1 || heads % cache->kv_heads || q_stride_seq < 0 || q_stride_node < 0 ||
      q_stride_head < 0 || stride_parents < 0 || !fp32_scale(scale) ||
      static_cast<int64_t>(cache->batch) * nodes * heads > kMaxRows)
    return TF_ERR_SHAPE;
  // The places of all items are numbered in 31 bits: a tile has 32 slots at least, and an item one place more.
  const int64_t tiles = (static_cast<int64_t>(cache->table_width) * cache->page_size + 31) / 32 + 2;
  if (static_cast<double>(tiles) * cache->kv_heads * cache->batch > 2147483647.0) return TF_ERR_SHAPE;
  if (dtype != TF_F16 && dtype != TF_BF16) return TF_ERR_DTYPE;
  if (cache->batch == 0 || nodes == 0) return TF_OK;
  s = check_cache_pointers(cache);
  if (s == TF_ERR_NULL || !q || !parents || !out || !lse || !workspace) return TF_ERR_NULL;
  if (s != TF_OK || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(parents, 4) ||
      !aligned(workspace, 256) || !eights(q_stride_seq, q_stride_node, q_stride_head))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  s = current_device_state(&device, &sms, &err);
  if (s == TF_OK) s = check_cache_device(cache, device);
  if (s == TF_OK) s = check_pointers_on_device(device, {q, parents, out, lse, workspace});
  if (s != TF_OK) return s;
  const AttendWorkspace ws = kvq_attend_workspace(nodes, heads, cache->kv_heads, cache->head_dim, sms);
  if (workspace_bytes < ws.bytes) return TF_ERR_SCRATCH;
  const QView view = view_of(cache, err);
  QAttendArgs x;
  x.scale_page = view.scale_page;
  x.scale_token = view.scale_token;
  x.scale_head = view.scale_head;
  x.scales = view.scales;
  x.box = 0;
  AttendArgs& a = x.a;
  a.c = view.c;
  a.k = cache->k;
  a.v = cache->v;
  a.q = q;
  a.q_seq = q_stride_seq;
  a.q_node = q_stride_node;
  a.q_head = q_stride_head;
  a.parents = parents;
  a.stride_parents = stride_parents;
  a.out = out;
  a.lse = lse;
  a.nodes = nodes;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.scale = static_cast<float>(scale);
  a.counters = static_cast<int*>(workspace);
  a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.partials_at);
  a.num_sms = sms;
  a.join_later = 0;
  return launched(launch_kvq_attention(x, dtype, cache->bits, device, static_cast<cudaStream_t>(stream)),
                  "quantised cache attention launch");
}

tf_status tf_kvq_keep(const tf_kvq_cache* cache, const int32_t* path, const int32_t* counts, int nodes,
                      int32_t* new_lengths, void* stream) {
  tf_status s = check_cache(cache, nodes);
  if (s != TF_OK) return s;
  if (cache->batch == 0) return TF_OK;
  if (nodes == 0) return TF_ERR_SHAPE;
  s = check_cache_pointers(cache);
  if (s == TF_ERR_NULL || !path || !counts || !new_lengths) return TF_ERR_NULL;
  if (s != TF_OK || !aligned(path, 4) || !aligned(counts, 4) || !aligned(new_lengths, 4)) return TF_ERR_ALIGN;
  // One block of a sequence writes its new length while others still read these.
  const int64_t batch = cache->batch;
  if (overlap(new_lengths, batch, cache->lengths, batch) || overlap(new_lengths, batch, counts, batch) ||
      overlap(new_lengths, batch, path, batch * nodes) ||
      overlap(new_lengths, batch, cache->page_table, (batch - 1) * cache->stride_table + cache->table_width))
    return TF_ERR_POINTER;
  int device, sms, *err;
  s = current_device_state(&device, &sms, &err);
  if (s == TF_OK) s = check_cache_device(cache, device);
  if (s == TF_OK) s = check_pointers_on_device(device, {path, counts, new_lengths});
  if (s != TF_OK) return s;
  return launched(launch_kvq_keep(view_of(cache, err), path, counts, nodes, new_lengths,
                                  static_cast<cudaStream_t>(stream)),
                  "quantised cache keep launch");
}

}  // extern "C"
