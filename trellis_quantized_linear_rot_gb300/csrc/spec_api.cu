// C ABI of the operators declared in tf_spec.h: argument checks, then a launch
// on the caller's stream.
#include <cmath>
#include <cstring>
#include <limits>

#include "spec.h"

using namespace tfx;

namespace {

constexpr int kMaxVocab = 1 << 24;
constexpr int64_t kMaxRows = int64_t{1} << 24;  // batch * nodes * heads of one call

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool eights(int64_t a, int64_t b, int64_t c) { return ((a | b | c) & 7) == 0; }

// Whether two arrays of 32-bit numbers share any.
bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uint64_t>(nb) * 4 && y < x + static_cast<uint64_t>(na) * 4;
}

// Whether the factor of a score is a number in fp32 (false for NaN).
bool fp32_scale(double scale) {
  return std::fabs(scale) <= std::numeric_limits<float>::max() && std::isfinite(static_cast<float>(scale) * kLog2e);
}

// The checks of a cache that need no device; *view and the device's state on TF_OK.
tf_status check_cache(const tf_kv_cache* c, int nodes) {
  if (!c) return TF_ERR_NULL;
  if (c->batch < 0 || nodes < 0 || nodes > TF_MAX_NODES || c->layers < 1 || c->pages < 1 || c->page_size < 1 ||
      c->kv_heads < 1 || c->head_dim < 8 || c->head_dim % 8 || c->head_dim > 1024 || c->table_width < 1)
    return TF_ERR_SHAPE;
  if (c->batch > 65535 || c->layers > 65535 || c->kv_heads > 65535 ||
      static_cast<int64_t>(c->table_width) * c->page_size > INT32_MAX - 2 * TF_MAX_NODES)
    return TF_ERR_SHAPE;
  if (c->stride_layer < 0 || c->stride_page < 0 || c->stride_token < 0 || c->stride_head < 0 || c->stride_table < 0)
    return TF_ERR_SHAPE;
  if (c->dtype != TF_F16 && c->dtype != TF_BF16) return TF_ERR_DTYPE;
  return TF_OK;
}

tf_status check_cache_pointers(const tf_kv_cache* c) {
  if (!c->k || !c->v || !c->page_table || !c->lengths) return TF_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) || !aligned(c->lengths, 4) ||
      !eights(c->stride_layer, c->stride_page, c->stride_token) || (c->stride_head & 7))
    return TF_ERR_ALIGN;
  return TF_OK;
}

CacheView view_of(const tf_kv_cache* c, int* err) {
  CacheView v;
  v.stride_layer = c->stride_layer;
  v.stride_page = c->stride_page;
  v.stride_token = c->stride_token;
  v.stride_head = c->stride_head;
  v.page_table = c->page_table;
  v.lengths = c->lengths;
  v.stride_table = c->stride_table;
  v.layers = c->layers;
  v.pages = c->pages;
  v.page_size = c->page_size;
  v.kv_heads = c->kv_heads;
  v.head_dim = c->head_dim;
  v.batch = c->batch;
  v.table_width = c->table_width;
  v.by_page = FastDiv(static_cast<uint32_t>(c->page_size));
  v.err = err;
  return v;
}

tf_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TF_OK : record_cuda_error(e, what); }

}  // namespace

extern "C" {

tf_status tf_kv_write(const tf_kv_cache* cache, const void* k_new, const void* v_new, int64_t stride_seq,
                      int64_t stride_node, int64_t stride_head, int nodes, void* stream) {
  tf_status s = check_cache(cache, nodes);
  if (s != TF_OK) return s;
  if (cache->layers != 1 || stride_seq < 0 || stride_node < 0 || stride_head < 0) return TF_ERR_SHAPE;
  if (cache->batch == 0 || nodes == 0) return TF_OK;
  s = check_cache_pointers(cache);
  if (s == TF_ERR_NULL || !k_new || !v_new) return TF_ERR_NULL;
  if (s != TF_OK || !aligned(k_new, 16) || !aligned(v_new, 16) || !eights(stride_seq, stride_node, stride_head))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  s = current_device_state(&device, &sms, &err);
  if (s == TF_OK)
    s = check_pointers_on_device(device, {cache->k, cache->v, cache->page_table, cache->lengths, k_new, v_new});
  if (s != TF_OK) return s;
  return launched(launch_kv_write(view_of(cache, err), cache->k, cache->v, k_new, v_new, stride_seq, stride_node,
                                  stride_head, nodes, static_cast<cudaStream_t>(stream)),
                  "cache write launch");
}

tf_status tf_kv_keep(const tf_kv_cache* cache, const int32_t* path, const int32_t* counts, int nodes,
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
  if (s == TF_OK)
    s = check_pointers_on_device(
        device, {cache->k, cache->v, cache->page_table, cache->lengths, path, counts, new_lengths});
  if (s != TF_OK) return s;
  return launched(launch_kv_keep(view_of(cache, err), cache->k, cache->v, path, counts, nodes, new_lengths,
                                 static_cast<cudaStream_t>(stream)),
                  "cache keep launch");
}

size_t tf_tree_attention_workspace_bytes(int batch, int nodes, int heads, int kv_heads, int head_dim) {
  if (batch < 0 || batch > 65535 || nodes < 0 || nodes > TF_MAX_NODES || heads < 1 || kv_heads < 1 ||
      heads % kv_heads || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  int device, sms, *err;
  if (current_device_state(&device, &sms, &err) != TF_OK) return 0;
  return attend_workspace(nodes, heads, kv_heads, head_dim, sms).bytes;
}

tf_status tf_tree_attention(const tf_kv_cache* cache, const void* q, int64_t q_stride_seq, int64_t q_stride_node,
                            int64_t q_stride_head, const int32_t* parents, int64_t stride_parents, void* out,
                            float* lse, int nodes, int heads, double scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
  tf_status s = check_cache(cache, nodes);
  if (s != TF_OK) return s;
  const int d = cache->head_dim;
  if (cache->layers != 1 || heads < 1 || heads % cache->kv_heads || (d != 64 && d != 128 && d != 256) ||
      q_stride_seq < 0 || q_stride_node < 0 || q_stride_head < 0 || stride_parents < 0 || !fp32_scale(scale) ||
      static_cast<int64_t>(cache->batch) * nodes * heads > kMaxRows)
    return TF_ERR_SHAPE;
  // The kernels number the places of all items in 31 bits. With mma.sync an item has a place for each tile
  // of 32 slots at least, and one more; on tcgen05 one for each tile of 128 and four more, which is no more
  // than counted here from 65 slots on, and 5 for each of kMaxRows items at most below.
  const int64_t tiles = (static_cast<int64_t>(cache->table_width) * cache->page_size + 31) / 32 + 2;
  if (static_cast<double>(tiles) * cache->kv_heads * cache->batch > 2147483647.0)
    return TF_ERR_SHAPE;
  if (cache->batch == 0 || nodes == 0) return TF_OK;
  s = check_cache_pointers(cache);
  if (s == TF_ERR_NULL || !q || !parents || !out || !lse || !workspace) return TF_ERR_NULL;
  if (s != TF_OK || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(parents, 4) ||
      !aligned(workspace, 256) || !eights(q_stride_seq, q_stride_node, q_stride_head))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  s = current_device_state(&device, &sms, &err);
  if (s == TF_OK)
    s = check_pointers_on_device(
        device, {cache->k, cache->v, cache->page_table, cache->lengths, q, parents, out, lse, workspace});
  if (s != TF_OK) return s;
  const AttendWorkspace ws = attend_workspace(nodes, heads, cache->kv_heads, d, sms);
  if (workspace_bytes < ws.bytes) return TF_ERR_SCRATCH;
  AttendArgs a;
  a.c = view_of(cache, err);
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
  return launched(launch_tree_attention(a, cache->dtype, device, static_cast<cudaStream_t>(stream)),
                  "tree attention launch");
}

size_t tf_verify_draft_workspace_bytes(int batch, int nodes) {
  if (batch < 0 || batch > 65535 || nodes < 1 || nodes > TF_MAX_NODES) return 0;
  int device, sms, *err;
  if (current_device_state(&device, &sms, &err) != TF_OK) return 0;
  return verify_workspace_bytes(batch, nodes, sms);
}

tf_status tf_verify_draft(const void* logits, int dtype, int64_t stride_seq, int64_t stride_node,
                          const void* draft_logits, int64_t draft_stride_seq, int64_t draft_stride_node,
                          const int32_t* tokens, const int32_t* parents, int64_t stride_parents,
                          const float* u_accept, const float* u_sample, double temperature, int batch, int nodes,
                          int vocab, int32_t* counts, int32_t* path, int32_t* out_tokens, float* logprobs,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || batch > 65535 || nodes < 1 || nodes > TF_MAX_NODES || vocab < 1 || vocab > kMaxVocab ||
      stride_seq < 0 || stride_node < 0 || draft_stride_seq < 0 || draft_stride_node < 0 || stride_parents < 0 ||
      !(temperature >= 0.0) || !std::isfinite(temperature) ||
      (temperature > 0.0 &&
       !(1.0 / temperature <= std::numeric_limits<float>::max() && static_cast<float>(1.0 / temperature) > 0.f)))
    return TF_ERR_SHAPE;
  if (dtype != TF_F16 && dtype != TF_F32 && dtype != TF_BF16) return TF_ERR_DTYPE;
  if (batch == 0) return TF_OK;
  const bool greedy = temperature == 0.0;
  const bool draft = draft_logits != nullptr && !greedy;
  if (!logits || !tokens || !parents || (!greedy && !u_sample) || (draft && !u_accept) || !counts || !path ||
      !out_tokens || !logprobs || !workspace)
    return TF_ERR_NULL;
  const uintptr_t elem = dtype == TF_F32 ? 4 : 2;
  if (!aligned(logits, elem) || !aligned(draft_logits, elem) || !aligned(tokens, 4) || !aligned(parents, 4) ||
      !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(counts, 4) || !aligned(path, 4) ||
      !aligned(out_tokens, 4) || !aligned(logprobs, 4) || !aligned(workspace, 256))
    return TF_ERR_ALIGN;
  int device, sms, *err;
  tf_status s = current_device_state(&device, &sms, &err);
  if (s == TF_OK)
    s = check_pointers_on_device(device,
                                 {logits, tokens, parents, workspace, counts, path, out_tokens, logprobs});
  if (s == TF_OK && !greedy) s = check_pointers_on_device(device, {u_sample});
  if (s == TF_OK && draft) s = check_pointers_on_device(device, {u_accept, draft_logits});
  if (s != TF_OK) return s;
  if (workspace_bytes < verify_workspace_bytes(batch, nodes, sms)) return TF_ERR_SCRATCH;
  VerifyArgs a;
  a.logits = logits;
  a.draft = draft ? draft_logits : nullptr;
  a.seq = stride_seq;
  a.node = stride_node;
  a.draft_seq = draft_stride_seq;
  a.draft_node = draft_stride_node;
  a.tokens = tokens;
  a.parents = parents;
  a.stride_parents = stride_parents;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.inv_temp = greedy ? 1.f : static_cast<float>(1.0 / temperature);
  a.greedy = greedy;
  a.batch = batch;
  a.nodes = nodes;
  a.vocab = vocab;
  a.counts = counts;
  a.path = path;
  a.out_tokens = out_tokens;
  a.logprobs = logprobs;
  a.work = static_cast<int*>(workspace);
  a.err = err;
  a.num_sms = sms;
  return launched(launch_verify_draft(a, dtype, static_cast<cudaStream_t>(stream)), "draft verification launch");
}

}  // extern "C"
