/*
 * tf_spec.h -- C ABI of the operators between the decode-row projections of
 * tf_exl3.h when several rows of a pass belong to one sequence: a tree of
 * drafted tokens is written into a paged cache (tf_kv_write), attends to it
 * (tf_tree_attention), its logits are checked against the target's
 * probabilities (tf_verify_draft), and the accepted path is kept
 * (tf_kv_keep). A tree of one node is the ordinary decode of one token.
 *
 * Conventions are those of tf_exl3.h: device pointers owned by the caller,
 * asynchronous calls on `stream`, arguments checked before any launch, no
 * call traps. Strides are in elements. Index arrays are int32. What a call
 * writes must overlap nothing that it reads (the cache of tf_kv_keep aside).
 *
 * A sequence's tree has `nodes` nodes (at most TF_MAX_NODES). Node 0 is the
 * last accepted token; the others are drafted. parents[j] is the parent of
 * node j: -1 for a node without one, otherwise less than j; -2 or less marks
 * an absent node (padding). Node i's key and value sit in slot
 * lengths[b] + i of the sequence, after its lengths[b] context tokens. A
 * negative length marks an idle sequence: nothing of it is read or written
 * (its output rows are those of absent nodes).
 *
 * Indices live on the device, so the host cannot check them. The kernels do:
 * an index outside its array (a page, a slot past the table, a parent or a
 * path entry out of order) is skipped, never followed, and recorded; the
 * next tf_device_error returns TF_ERR_INDEX.
 */
#ifndef TF_SPEC_H
#define TF_SPEC_H

#include "tf_exl3.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { TF_MAX_NODES = 128 };

/* A paged cache and the sequences that use it. Slot s of sequence b is row
 * s % page_size of page page_table[b * stride_table + s / page_size]; head h
 * of that row starts at layer * stride_layer + page * stride_page + row *
 * stride_token + h * stride_head, and its head_dim elements are contiguous.
 * k and v share the strides. Every stride is a multiple of 8 elements, k and
 * v are 16-byte aligned, head_dim is a multiple of 8. */
typedef struct {
  void* k;
  void* v;
  int64_t stride_layer, stride_page, stride_token, stride_head;
  const int32_t* page_table; /* [batch][table_width], rows stride_table apart */
  const int32_t* lengths;    /* [batch] */
  int64_t stride_table;
  int32_t dtype;             /* TF_F16 or TF_BF16 */
  int32_t layers, pages, page_size, kv_heads, head_dim;
  int32_t batch, table_width;
} tf_kv_cache;

/*
 * tf_kv_write -- writes the keys and values of a tree's nodes into the cache:
 *   k[slot lengths[b] + i][h] = k_new[b][i][h], and v likewise, i < nodes.
 * k_new, v_new: [batch][nodes][kv_heads][head_dim] of the cache's dtype, with
 * the given strides (a part of a fused projection's rows, for example), the
 * last dimension contiguous; 16-byte aligned, strides multiples of 8.
 * cache->layers must be 1. The pages have no counterpart.
 */
tf_status tf_kv_write(const tf_kv_cache* cache, const void* k_new, const void* v_new,
                      int64_t stride_seq, int64_t stride_node, int64_t stride_head, int nodes,
                      void* stream);

/*
 * tf_tree_attention -- attention of a tree's nodes over the cache. Row
 * (b, i, h) sees the context slots 0 .. lengths[b]-1 and the slots of node i
 * and its ancestors:
 *   s = scale * (q . k) over the seen slots, in fp32
 *   out = sum exp(s - max s) v / sum exp(s - max s), rounded once to the dtype
 *   lse = max s + log sum exp(s - max s), fp32, natural logarithm
 * A row that sees nothing (an absent node, an idle sequence) gets out = 0
 * and lse = -inf. What a row does not see has no influence on it, whatever
 * its bits (NaN and infinities among them).
 * The weights exp(s - max s) are rounded to the dtype for the second matrix
 * product; maxima, sums and accumulators are fp32.
 * q: [batch][nodes][heads][head_dim] with the given strides, last dimension
 *   contiguous, 16-byte aligned, strides multiples of 8. heads is a multiple
 *   of kv_heads; head h reads kv head h / (heads / kv_heads).
 * parents: [batch][nodes], rows stride_parents apart (0: one tree for all).
 * out: [batch][nodes][heads][head_dim] contiguous; lse: [batch][nodes][heads].
 * head_dim 64, 128 or 256; cache->layers must be 1. scale * log2(e) must be
 *   finite in fp32 (TF_ERR_SHAPE).
 * workspace: device memory, 256-byte aligned, at least
 *   tf_tree_attention_workspace_bytes(...) bytes, zeroed before its first use;
 *   each call leaves it ready for the next. Calls that share a workspace must
 *   be ordered by the caller. After TF_ERR_TIMEOUT it has to be zeroed again.
 * The same inputs give the same bits. The pages have no counterpart.
 */
tf_status tf_tree_attention(const tf_kv_cache* cache, const void* q, int64_t q_stride_seq,
                            int64_t q_stride_node, int64_t q_stride_head, const int32_t* parents,
                            int64_t stride_parents, void* out, float* lse, int nodes, int heads,
                            double scale, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace tf_tree_attention needs for these sizes on the current
 * device, 0 for sizes it refuses. Smaller sizes need no more, but for
 * kv_heads: fewer of them have more rows each, and one has the most. The
 * pages have no counterpart. */
size_t tf_tree_attention_workspace_bytes(int batch, int nodes, int heads, int kv_heads, int head_dim);

/*
 * tf_verify_draft -- which drafted tokens the target accepts, and the token
 * that follows them. Row (b, j) of `logits` is the target's prediction after
 * node j. From node 0 the call goes down the tree while a child is accepted,
 * then samples one more token at the node it ended on.
 * Probabilities: z = fp32(logit) * fp32(1 / temperature) (the factor must be
 * finite and above 0, else TF_ERR_SHAPE; a NaN z counts as -inf), e =
 * exp(z - max z) in fp32, w = round(2^30 e), P = sum w: whole numbers, so that
 * no order of summation changes a token.
 *   temperature 0: the next token is the largest logit's, lowest index first
 *     (probabilities as for temperature 1; u_sample, draft_logits unused).
 *   without draft_logits: the token at a node is the least i with
 *     w[0] + .. + w[i] > floor(u_sample[b][node] * P); the node's first child
 *     with that token is accepted.
 *   with draft_logits (row (b, j): the distribution the children of node j
 *     were drawn from, independently; same temperature; its f, Q as e, P):
 *     in units of 2^-31, p = e * fp32(2^61/P), q = f * fp32(2^61/Q). Children
 *     are asked in index order with a = 0, S = 2^31, r = p at first: child c
 *     with token t is accepted if u_accept[b][c] * q[t] * S < r[t] * 2^31 (in
 *     fp64); a refusal makes a += S/2^31, r = max(round(p) - round(f *
 *     fp32(a * 2^61/Q)), 0) and S = sum r, so that r/S is the normalised rest
 *     of the distribution. With S = 0 no more children are asked and r is p
 *     again. After the last refusal the token is the least i with r[0] + .. +
 *     r[i] > floor(u_sample[b][node] * S) (w and P where no child was refused).
 * What whole numbers leave out: a token whose e is below 2^-31 has no weight
 *   and is never sampled; P and the log-probabilities are off by up to vocab *
 *   2^-31 of themselves (6e-5 at 131072, 0.8 % at 2^24). After a refusal the
 *   unit is 2^-31 of p still, and so 1/S of what is left.
 * A child whose token lies outside [0, vocab) is passed over.
 * logits, draft_logits: [batch][nodes][vocab] of one dtype (TF_F32, TF_F16 or
 *   TF_BF16) with the given strides, last dimension contiguous; vocab <= 2^24.
 * tokens, u_accept, u_sample: [batch][nodes] (tokens[b][0], u_accept[b][0]
 *   unused), u in [0, 1). Other values are clamped, u_sample to the last token
 *   of its sum, u_accept to 1 (which refuses a child unless r[t] * 2^31 is
 *   above q[t] * S); a NaN counts as 0. parents as in tf_tree_attention.
 * Written, each [batch][nodes] unless said: counts [batch] = kept nodes (0
 *   for a sequence whose node 0 is absent); path: the kept nodes, first node
 *   0, then -1; out_tokens: the accepted tokens and the sampled one (-1 where
 *   no logit of its row is above -inf), then -1; logprobs fp32: their target
 *   log-probabilities at `temperature` (at 1 for temperature 0), then 0.
 * workspace as in tf_tree_attention, of tf_verify_draft_workspace_bytes.
 * The pages have no counterpart.
 */
tf_status tf_verify_draft(const void* logits, int dtype, int64_t stride_seq, int64_t stride_node,
                          const void* draft_logits, int64_t draft_stride_seq, int64_t draft_stride_node,
                          const int32_t* tokens, const int32_t* parents, int64_t stride_parents,
                          const float* u_accept, const float* u_sample, double temperature, int batch,
                          int nodes, int vocab, int32_t* counts, int32_t* path, int32_t* out_tokens,
                          float* logprobs, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace tf_verify_draft needs for these sizes and any smaller
 * ones, 0 for sizes it refuses. The pages have no counterpart. */
size_t tf_verify_draft_workspace_bytes(int batch, int nodes);

/*
 * tf_kv_keep -- keeps the accepted path in the cache, in every layer:
 *   slot lengths[b] + k = slot lengths[b] + path[b][k], k < counts[b],
 *   new_lengths[b] = lengths[b] + counts[b].
 * path: [batch][nodes], strictly rising and below nodes over its first
 * counts[b] entries (a path of tf_verify_draft); it is followed as far as it
 * is, and the rest recorded as TF_ERR_INDEX. new_lengths must not overlap
 * cache->lengths, cache->page_table, path or counts (TF_ERR_POINTER): every
 * block of the launch reads those. An idle sequence keeps its length. The
 * pages have no counterpart.
 */
tf_status tf_kv_keep(const tf_kv_cache* cache, const int32_t* path, const int32_t* counts, int nodes,
                     int32_t* new_lengths, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TF_SPEC_H */
