// Norms of queries and keys for each head, the rotation by their positions
// and the Hadamard rotation over the head, in one pass (tf_qk_norm_rope).
//
// head_dim / 8 lanes have a row, 8 elements each, in registers from the load
// to the store: the mean square is summed over the lanes by shuffles, the
// other half of a pair comes from the lane rotary / 16 away, and the Hadamard
// rotation is log2(head_dim) additions an element. A block takes heads of one
// token, whose cosines and sines it works out once for all of them. Reading
// and writing each row once is what bounds it; for few tokens the launch.
#include "qcache.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 256;
constexpr double kTurn = 0.15915494309189533577;   // 1 / (2 pi)

template <typename W>
__device__ __forceinline__ void load_weight(const void* weight, int at, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = weight ? to_f32(static_cast<const W*>(weight)[at + i]) : 1.f;
}

template <typename T, typename W, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int splits) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  __shared__ float2 turn[D / 2];   // cosine and sine of pair i
  chain();
  const int64_t token = blockIdx.x / splits;
  const int split = static_cast<int>(blockIdx.x - token * splits);
  const int b = static_cast<int>(token / a.nodes), node = static_cast<int>(token - static_cast<int64_t>(b) * a.nodes);
  const int pos = a.positions[b * a.stride_positions + node];
  if (pos < 0) return;
  const int half = a.rotary / 2;
  for (int i = threadIdx.x; i < half; i += kThreads) {
    // The angle in turns; whole turns are dropped in fp64.
    const double t = pos * a.inv_freq[i] * kTurn;
    float s, c;
    sincospif(static_cast<float>(2.0 * (t - rint(t))), &s, &c);
    turn[i] = float2{c, s};
  }
  __syncthreads();
  const int lane = threadIdx.x % kLanes, e = lane * 8;
  const bool interleaved = a.flags & TF_QK_INTERLEAVED;
  const int all = a.q.heads + a.k.heads;
  // Whole warps run through the loop together, so that lanes can meet.
  for (int r0 = split * kRows; r0 < all; r0 += splits * kRows) {
    const int r = min(r0 + static_cast<int>(threadIdx.x) / kLanes, all - 1);
    const bool key = r >= a.q.heads;
    const tf_head_rows& rows = key ? a.k : a.q;
    const int h = key ? r - a.q.heads : r;
    float x[8], w[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(rows.x) + b * rows.x_seq + node * rows.x_node +
                                               h * rows.x_head + e),
               x);
    load_weight<W>(rows.weight, e, w);
    if (!(a.flags & TF_QK_NO_NORM)) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
#pragma unroll
      for (int o = 1; o < kLanes; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
      const float f = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= w[i];
    if (half > 0 && interleaved) {
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        if (e + i < a.rotary) {
          const float2 t = turn[(e + i) / 2];
          const float u = x[i], v = x[i + 1];
          x[i] = u * t.x - v * t.y;
          x[i + 1] = v * t.x + u * t.y;
        }
    } else if (half > 0) {
      const bool first = e < half, turned = e < a.rotary;
      const int other = !turned ? lane : first ? lane + half / 8 : lane - half / 8;
      const int base = static_cast<int>(threadIdx.x % 32) - lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __shfl_sync(~0u, x[i], base + other);
        if (turned) {
          const float2 t = turn[first ? e + i : e + i - half];
          x[i] = x[i] * t.x + (first ? -v : v) * t.y;
        }
      }
    }
    if (a.flags & TF_QK_HADAMARD) {
#pragma unroll
      for (int o = 1; o < 8; o *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & o)) {
            const float u = x[i], v = x[i + o];
            x[i] = u + v;
            x[i + o] = u - v;
          }
#pragma unroll
      for (int o = 1; o < kLanes; o *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = __shfl_xor_sync(~0u, x[i], o);
          x[i] = lane & o ? v - x[i] : x[i] + v;
        }
      constexpr float f = D == 64 ? 0.125f : D == 128 ? 0.0883883476f : 0.0625f;   // 1 / sqrt(D)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= f;
    }
    if (r0 + static_cast<int>(threadIdx.x) / kLanes < all)
      *reinterpret_cast<uint4*>(static_cast<T*>(rows.y) + b * rows.y_seq + node * rows.y_node + h * rows.y_head + e) =
          pack8<T>(x);
  }
}

template <typename T, typename W>
cudaError_t launch(const NormRopeArgs& a, int head_dim, cudaStream_t s) {
  const int per = kThreads / (head_dim / 8), all = a.q.heads + a.k.heads;
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.nodes;
  // Few tokens: a block for each kThreads / lanes heads; many: one a token.
  const int splits = tokens < 4 * a.num_sms ? (all + per - 1) / per : 1;
  const dim3 grid(static_cast<unsigned>(tokens * splits));
  switch (head_dim) {
    case 64: return launch_chained(qk_norm_rope_kernel<T, W, 64>, grid, dim3(kThreads), 0, 1, s, a, splits);
    case 128: return launch_chained(qk_norm_rope_kernel<T, W, 128>, grid, dim3(kThreads), 0, 1, s, a, splits);
    default: return launch_chained(qk_norm_rope_kernel<T, W, 256>, grid, dim3(kThreads), 0, 1, s, a, splits);
  }
}

template <typename T>
cudaError_t by_weight(const NormRopeArgs& a, int weight_dtype, int head_dim, cudaStream_t s) {
  return weight_dtype == TF_F32   ? launch<T, float>(a, head_dim, s)
         : weight_dtype == TF_F16 ? launch<T, __half>(a, head_dim, s)
                                  : launch<T, __nv_bfloat16>(a, head_dim, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int dtype, int weight_dtype, int head_dim, cudaStream_t s) {
  return dtype == TF_F16 ? by_weight<__half>(a, weight_dtype, head_dim, s)
                         : by_weight<__nv_bfloat16>(a, weight_dtype, head_dim, s);
}

}  // namespace tfx
