// Attention of a drafted token tree over a quantised paged cache
// (tf_kvq_attention): a block of 128 threads for each row.
#include "attend_work.cuh"
#include "qcache.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 128;

template <typename T, int kBits, int D>
__global__ void __launch_bounds__(kThreads) kvq_attention_kernel(const __grid_constant__ QAttendArgs args) {
  const AttendArgs& a = args.a;
  __shared__ float q[D], weight[kThreads];
  __shared__ int64_t values_at[kThreads];
  __shared__ uint32_t seen[TF_MAX_NODES / 32];
  __shared__ float red[kThreads / 32];
  chain();
  const int head = blockIdx.x % a.heads, tid = threadIdx.x;
  const int node = blockIdx.x / a.heads % a.nodes, b = blockIdx.x / a.heads / a.nodes;
  const int kvh = head / a.group;
  const Span span = sequence_span(a.c, b, a.nodes);
  if (tid < TF_MAX_NODES / 32) seen[tid] = 0;
  for (int i = tid; i < D; i += kThreads)
    q[i] = to_f32(static_cast<const T*>(a.q)[b * a.q_seq + node * a.q_node + head * a.q_head + i]);
  __syncthreads();
  if (tid == 0) {
    for (int i = node; i >= 0;) {
      const int up = a.parents[b * a.stride_parents + i];
      if (up >= i) record_index_error(a.c.err);
      if (up >= i || up < -1) break;
      seen[i / 32] |= 1u << (i % 32);
      i = up;
    }
  }
  __syncthreads();
  const bool present = span.context >= 0 && (seen[node / 32] >> (node % 32) & 1);
  constexpr int kRow = D * kBits / 8;
  float m = -INFINITY, l = 0.f, o[(D + kThreads - 1) / kThreads] = {};
  for (int s0 = 0; present && s0 < span.slots; s0 += kThreads) {
    const int slot = s0 + tid, j = slot - span.context;
    Place at;
    float s = -INFINITY, factor = 0.f;
    int64_t place = 0;
    if (slot < span.slots && (j < 0 || (seen[j / 32] >> (j % 32) & 1)) && place_of(a.c, b, slot, &at)) {
      place = codes_at(a.c, at) + kvh * a.c.stride_head;
      const uint32_t w = args.scales[at.page * args.scale_page + at.row * args.scale_token + kvh * args.scale_head];
      const uint8_t* k = static_cast<const uint8_t*>(a.k) + place;
      float dot = 0.f;
      for (int i = 0; i < kRow; ++i) {
        if (kBits == 8) dot += q[i] * (k[i] - 128);
        else dot += q[2 * i] * ((k[i] & 15) - 8) + q[2 * i + 1] * ((k[i] >> 4) - 8);
      }
      s = dot * key_scale(w) * (a.scale * kLog2e);
      factor = value_scale(w);
    }
    float top = s;
    for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
    __syncthreads();
    if (tid % 32 == 0) red[tid / 32] = top;
    values_at[tid] = place;
    __syncthreads();
    top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = top == -INFINITY ? 0.f : top, keep = exp2_approx(m - base);
    const float p = s == -INFINITY ? 0.f : exp2_approx(s - base);
    m = top;
    weight[tid] = s == -INFINITY ? 0.f : p * factor;
    float sum = p;
    for (int x = 16; x; x /= 2) sum += __shfl_xor_sync(~0u, sum, x);
    __syncthreads();
    if (tid % 32 == 0) red[tid / 32] = sum;
    __syncthreads();
    l = l * keep + red[0] + red[1] + red[2] + red[3];
    for (int x = 0; x < (D + kThreads - 1) / kThreads; ++x) {
      const int e = x * kThreads + tid;
      if (e >= D) continue;
      float y = o[x] * keep;
      for (int i = 0; i < min(kThreads, span.slots - s0); ++i) {
        if (weight[i] == 0.f) continue;
        const uint8_t* v = static_cast<const uint8_t*>(a.v) + values_at[i];
        y += weight[i] * (kBits == 8 ? v[e] - 128 : (v[e / 2] >> (e % 2 * 4) & 15) - 8);
      }
      o[x] = y;
    }
  }
  const bool empty = !present || l == 0.f;
  const size_t row = blockIdx.x;
  for (int x = 0; x < (D + kThreads - 1) / kThreads; ++x) {
    const int e = x * kThreads + tid;
    if (e < D) static_cast<T*>(a.out)[row * D + e] = from_f32<T>(empty ? 0.f : o[x] / l);
  }
  if (tid == 0) a.lse[row] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T, int kBits>
cudaError_t launch(const QAttendArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.a.c.batch) * a.a.nodes * a.a.heads), block(kThreads);
  switch (a.a.c.head_dim) {
    case 64: return launch_chained(kvq_attention_kernel<T, kBits, 64>, grid, block, 0, 1, s, a);
    case 128: return launch_chained(kvq_attention_kernel<T, kBits, 128>, grid, block, 0, 1, s, a);
    default: return launch_chained(kvq_attention_kernel<T, kBits, 256>, grid, block, 0, 1, s, a);
  }
}

}  // namespace

AttendWorkspace kvq_attend_workspace(int nodes, int heads, int kv_heads, int head_dim, int num_sms) {
  return attend_workspace(nodes, heads, kv_heads, head_dim, num_sms);
}

cudaError_t launch_kvq_attention(const QAttendArgs& a, int dtype, int bits, int device, cudaStream_t s) {
  (void)device;
  if (dtype == TF_F16) return bits == 4 ? launch<__half, 4>(a, s) : launch<__half, 8>(a, s);
  return bits == 4 ? launch<__nv_bfloat16, 4>(a, s) : launch<__nv_bfloat16, 8>(a, s);
}

}  // namespace tfx
