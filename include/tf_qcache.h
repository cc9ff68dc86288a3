/*
 * tf_qcache.h -- C ABI of the operators between the qkv projection and the
 * attention when the paged cache is held in 4 or 8 bits: queries and keys are
 * normed for each head and rotated by their positions (tf_qk_norm_rope), keys
 * and values are quantised as they are written (tf_kvq_write), read back
 * (tf_kvq_read), attended to (tf_kvq_attention), and the accepted path of a
 * drafted tree is kept (tf_kvq_keep).
 *
 * Conventions are those of tf_exl3.h and tf_spec.h: device pointers owned by
 * the caller, asynchronous calls on `stream`, arguments checked before any
 * launch, no call traps; trees, slots, idle sequences and the treatment of
 * indices outside their arrays (TF_ERR_INDEX from the next tf_device_error)
 * as in tf_spec.h. What a call writes must overlap nothing that it reads
 * unless said otherwise.
 */
#ifndef TF_QCACHE_H
#define TF_QCACHE_H

#include "tf_spec.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows of one kind (queries or keys) of tf_qk_norm_rope: x and y are
 * [batch][nodes][heads][head_dim] with the given strides in elements, the
 * last dimension contiguous; 16-byte aligned, strides multiples of 8. y may
 * be x itself with the same strides. weight: [head_dim], NULL for ones.
 */
typedef struct {
  const void* x;
  void* y;
  const void* weight;
  int64_t x_seq, x_node, x_head;
  int64_t y_seq, y_node, y_head;
  int32_t heads;
} tf_head_rows;

enum {
  TF_QK_NO_NORM = 1,      /* the rows are not divided by their root mean square */
  TF_QK_INTERLEAVED = 2,  /* pairs (2i, 2i+1) instead of (i, i + rotary/2) */
  TF_QK_HADAMARD = 4      /* a Hadamard rotation over the head at the end */
};

/*
 * tf_qk_norm_rope -- for each row x of a query or key head:
 *   u = weight * x / sqrt(mean(x^2) + eps)                 (fp32)
 *   (u[a], u[b]) = (u[a] cos t - u[b] sin t, u[b] cos t + u[a] sin t) over
 *     the pairs i < rotary/2 of its first `rotary` elements, t =
 *     positions[b][node] * inv_freq[i] (fp64, reduced to a turn before cos
 *     and sin, so that far positions lose nothing)
 *   y = u, or H u / sqrt(head_dim) with TF_QK_HADAMARD, H[i][j] = -1 to the
 *     number of ones that i and j have in common
 * rounded once to the dtype. Rows of any size are normed, those too whose
 * squares fp32 does not hold; with eps 0 a row of zeros is NaN. The last step
 * leaves q.k as it is and spreads large elements over the head before they
 * are quantised.
 * A negative position marks a row that is not there: what it holds has no
 * influence, and nothing is written. keys may be NULL (queries alone).
 * dtype: TF_F16 or TF_BF16; weight_dtype: also TF_F32. positions: [batch]
 * [nodes], rows stride_positions apart (0: one for all). inv_freq: fp64
 * [rotary/2]. rotary: a multiple of 16 up to head_dim, 0 for no rotation
 * (inv_freq unused). head_dim 64, 128 or 256. eps >= 0. The pages have no
 * counterpart.
 */
tf_status tf_qk_norm_rope(const tf_head_rows* queries, const tf_head_rows* keys, int dtype, int weight_dtype,
                          const int32_t* positions, int64_t stride_positions, const double* inv_freq, int rotary,
                          double eps, int flags, int batch, int nodes, int head_dim, void* stream);

/*
 * A paged cache of quantised rows and the sequences that use it. A row is the
 * key or value of one slot and head: head_dim whole numbers c and a factor s
 * (bf16); its values are c * s. |c| <= 7 with 4 bits (stored c + 8, element
 * 2i in the low half of byte i) and <= 127 with 8 (stored c + 128). Slot s of
 * sequence b is row s % page_size of page page_table[b * stride_table + s /
 * page_size]; its codes of head h start at layer * stride_layer + page *
 * stride_page + row * stride_token + h * stride_head of k and v (bytes,
 * multiples of 16; k and v share them, are 16-byte aligned), the factors of
 * key and value lie side by side at layer * scale_layer + ... of scales
 * (elements, multiples of 2; 4-byte aligned). Rows of one head and page that
 * lie together are read fastest. head_dim 64, 128 or 256.
 */
typedef struct {
  void* k;
  void* v;
  void* scales;
  int64_t stride_layer, stride_page, stride_token, stride_head;
  int64_t scale_layer, scale_page, scale_token, scale_head;
  const int32_t* page_table; /* [batch][table_width], rows stride_table apart */
  const int32_t* lengths;    /* [batch] */
  int64_t stride_table;
  int32_t bits;              /* 4 or 8 */
  int32_t layers, pages, page_size, kv_heads, head_dim;
  int32_t batch, table_width;
} tf_kvq_cache;

/*
 * tf_kvq_write -- quantises keys and values into slots lengths[b] + i:
 *   s = bf16(max |x| / m), c = round(x / s) to the nearest, ties to even,
 *   held to +-m; m = 7 or 127; c = 0 where s is 0. A row with an element that
 *   is not finite gets s = NaN and c = 0: it is NaN for whoever sees it.
 * k_new, v_new: [batch][nodes][kv_heads][head_dim] fp16 or bf16, each with
 * strides of its own (keys that were normed lie elsewhere than values of a
 * projection's rows), otherwise as in tf_kv_write. nodes is not limited to a tree's: parts
 * of prompts are written the same way (up to 2^31 rows in all). counts:
 * [batch], tokens of each sequence (the others are padding, not read), or
 * NULL for all. cache->layers must be 1. The pages have no counterpart.
 */
tf_status tf_kvq_write(const tf_kvq_cache* cache, const void* k_new, int64_t k_stride_seq, int64_t k_stride_node,
                       int64_t k_stride_head, const void* v_new, int64_t v_stride_seq, int64_t v_stride_node,
                       int64_t v_stride_head, int dtype, const int32_t* counts, int nodes, void* stream);

/*
 * tf_kvq_read -- the values of slots starts[b] + i, i < slots, below
 * lengths[b], each rounded once to the dtype: k_out, v_out: [batch][slots]
 * [kv_heads][head_dim] fp16 or bf16 with the given strides, last dimension
 * contiguous; 16-byte aligned, strides multiples of 8. c * s may be above a
 * row's largest element by 2^-9 of it (s is rounded), and infinite in fp16 for
 * elements next to its largest. Rows of other slots are left as they were.
 * starts: [batch], or NULL for 0. cache->layers must be 1. The pages have no
 * counterpart.
 */
tf_status tf_kvq_read(const tf_kvq_cache* cache, const int32_t* starts, void* k_out, void* v_out, int dtype,
                      int64_t stride_seq, int64_t stride_slot, int64_t stride_head, int slots, void* stream);

/*
 * tf_kvq_attention -- tf_tree_attention over the values of a quantised
 * cache: the same arguments, masks, outputs and refusals. q and out are fp16
 * or bf16 (dtype). Codes go into the matrix products as they are; the factors
 * of keys multiply scores in fp32, those of values the weights, which are
 * rounded for the second product: to 11 bits, and to 2^-26 of the row's
 * largest weight where they are smaller than 2^-15 of it. Weights exp(s - max
 * s) below 2^-126 are 0. Maxima, sums and accumulators are fp32, and scores may
 * have any size that fp32 holds. workspace as there, of
 * tf_kvq_attention_workspace_bytes; the two operators may share one that is
 * large enough for both.
 * The same inputs give the same bits. The pages have no counterpart.
 */
tf_status tf_kvq_attention(const tf_kvq_cache* cache, const void* q, int dtype, int64_t q_stride_seq,
                           int64_t q_stride_node, int64_t q_stride_head, const int32_t* parents,
                           int64_t stride_parents, void* out, float* lse, int nodes, int heads, double scale,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace tf_kvq_attention needs for these sizes on the current
 * device, 0 for sizes it refuses. Smaller sizes need no more, but for
 * kv_heads: fewer of them have more rows each, and one has the most. The
 * pages have no counterpart. */
size_t tf_kvq_attention_workspace_bytes(int batch, int nodes, int heads, int kv_heads, int head_dim);

/*
 * tf_kvq_keep -- tf_kv_keep for a quantised cache: codes and factors of the
 * accepted path moved together, in every layer; the same refusals. The pages
 * have no counterpart.
 */
tf_status tf_kvq_keep(const tf_kvq_cache* cache, const int32_t* path, const int32_t* counts, int nodes,
                      int32_t* new_lengths, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TF_QCACHE_H */
