// Attention of a drafted token tree over a paged cache (tf_tree_attention).
//
// One block takes one row (sequence, node, head) and walks the slots the row
// sees in tiles of 128, with the running maximum and sum of the softmax: one
// thread a slot for the scores, one thread a column for the weighted sum.
#include "spec.cuh"

namespace tfx {
namespace {

constexpr int kTile = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kTile) tree_attention_row_kernel(AttendArgs a) {
  __shared__ TreeMasks masks;
  __shared__ float qs[D], ps[kTile], red[4];
  __shared__ int64_t at[kTile];
  const CacheView& c = a.c;
  const int row = blockIdx.x, tid = threadIdx.x;
  const int h = row % a.heads, i = row / a.heads % a.nodes, b = row / a.heads / a.nodes;
  const int kvh = h / a.group;
  const T* q = static_cast<const T*>(a.q) + b * a.q_seq + i * a.q_node + h * a.q_head;
  const T* k = static_cast<const T*>(a.k) + kvh * c.stride_head;
  const T* v = static_cast<const T*>(a.v) + kvh * c.stride_head;
  for (int e = tid; e < D; e += kTile) qs[e] = to_f32(q[e]);
  build_tree_masks(masks, a.parents + b * a.stride_parents, a.nodes, c.err);
  const Span span = sequence_span(c, b, a.nodes);
  const int len = span.context;
  const bool present = len >= 0 && (masks.anc[i][i >> 5] >> (i & 31) & 1);
  float m = -INFINITY, l = 0.f, acc[(D + kTile - 1) / kTile] = {};
  const int total = present ? min(span.slots, len + i + 1) : 0;
  for (int s0 = 0; s0 < total; s0 += kTile) {
    const int s = s0 + tid, j = s - len;
    bool sees = s < total && (j < 0 || (masks.anc[i][j >> 5] >> (j & 31) & 1));
    at[tid] = sees ? slot_offset(c, b, s) : -1;
    sees = at[tid] >= 0;
    float x = -INFINITY;
    if (sees) {
      x = 0.f;
      for (int e = 0; e < D; ++e) x += qs[e] * to_f32(k[at[tid] + e]);
      x *= a.scale;
    }
    float top = x;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (tid % 32 == 0) red[tid / 32] = top;
    __syncthreads();
    const float m1 = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float keep = m == -INFINITY ? 0.f : expf(m - m1);
    const float p = x == -INFINITY ? 0.f : expf(x - m1);
    m = m1;
    ps[tid] = p;
    float sum = p;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    __syncthreads();
    if (tid % 32 == 0) red[tid / 32] = sum;
    __syncthreads();
    l = l * keep + (red[0] + red[1] + red[2] + red[3]);
    for (int n = 0; n * kTile < D; ++n) {
      const int e = n * kTile + tid;
      float y = acc[n] * keep;
      if (e < D)
        for (int t = 0; t < kTile; ++t)
          if (at[t] >= 0) y += ps[t] * to_f32(v[at[t] + e]);
      acc[n] = y;
    }
    __syncthreads();
  }
  T* out = static_cast<T*>(a.out) + static_cast<int64_t>(row) * D;
  for (int n = 0; n * kTile < D; ++n)
    if (n * kTile + tid < D) out[n * kTile + tid] = from_f32<T>(l > 0.f ? acc[n] / l : (l == 0.f ? 0.f : l));
  if (tid == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T>
cudaError_t launch_typed(const AttendArgs& a, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.c.batch) * a.nodes * a.heads;
  if (a.c.head_dim == 64) tree_attention_row_kernel<T, 64><<<rows, kTile, 0, s>>>(a);
  if (a.c.head_dim == 128) tree_attention_row_kernel<T, 128><<<rows, kTile, 0, s>>>(a);
  if (a.c.head_dim == 256) tree_attention_row_kernel<T, 256><<<rows, kTile, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attention(const AttendArgs& a, int dtype, cudaStream_t s) {
  return dtype == TF_F16 ? launch_typed<__half>(a, s) : launch_typed<__nv_bfloat16>(a, s);
}

}  // namespace tfx
