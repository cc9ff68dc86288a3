// Norms of queries and keys for each head, the rotation by their positions
// and the Hadamard rotation over the head, in one pass (tf_qk_norm_rope).
//
// head_dim / 16 lanes have a row, in registers from the load to the store: a
// lane the c-th 8 elements of each half of the head. So the pair of an element
// (half a head away where the whole head is rotated) is the same lane's, and
// the Hadamard rotation leaves the lane for log2(head_dim) - 4 of its steps. A
// block takes several tokens (as many as its threads can work out the cosines
// and sines of at once), whose rows follow one another; the next row is asked
// for before this one is worked on. Reading and writing each row once is what
// bounds it, and close to that the instructions, so two elements are worked on
// by one wherever they can be. For few tokens the launch.
// Measured: 4,096 tokens of 48 + 8 heads of 128 in bf16 37.7 us with the
// Hadamard rotation, 29.4 without (117 MB: 3.1 and 4.0 TB/s), issue slots 61%
// busy; 1 token of 40 + 8 heads 3.0 us. Lanes that stay with a token and have
// its cosines in registers have a quarter fewer instructions, but fewer warps:
// 34 to 39 us, and 300 tokens 7.4 to 9.3 for 6.4.
#include <algorithm>
#include <type_traits>

#include "qcache.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 256;
constexpr double kTurn = 0.15915494309189533577;   // 1 / (2 pi)

// Eight elements as four pairs.
template <typename T>
__device__ __forceinline__ void pairs_of(const uint4& w, float2 (&x)[4]) {
  float f[8];
  unpack8<T>(w, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = float2{f[2 * i], f[2 * i + 1]};
}
template <typename W>
__device__ __forceinline__ void load_weight(const void* weight, int at, float2 (&w)[4]) {
  if (!weight) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = float2{1.f, 1.f};
    return;
  }
  // (a weight is aligned to its type only)
  const W* p = static_cast<const W*>(weight) + at;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    if constexpr (sizeof(W) == 4) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      w[0] = float2{a.x, a.y}, w[1] = float2{a.z, a.w}, w[2] = float2{b.x, b.y}, w[3] = float2{b.z, b.w};
    } else {
      pairs_of<W>(*reinterpret_cast<const uint4*>(p), w);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) w[i] = float2{to_f32(p[2 * i]), to_f32(p[2 * i + 1])};
  }
}
__device__ __forceinline__ float2 twice(float x) { return float2{x, x}; }
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return fma2(b, twice(-1.f), a); }

template <typename T, typename W, int D>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int tokens, int per_block, int splits, FastDiv by_nodes,
                    FastDiv by_rows) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes, kHalf = D / 2;
  __shared__ __align__(16) float cosines[kThreads], sines[kThreads];   // of pair i of token k at k * half + i
  __shared__ int positions[kThreads];
  chain();
  const int split = blockIdx.x % splits, token0 = static_cast<int>(blockIdx.x / splits) * per_block;
  const int here = min(per_block, tokens - token0);   // tokens of this block
  const int half = a.rotary / 2;
  const int lane = threadIdx.x % kLanes, e = lane * 8, all = a.q.heads + a.k.heads, rows = here * all;
  struct Row {
    const tf_head_rows* kind;
    int k, b, node, head;   // k: its token's number in the block
  };
  auto row_of = [&](int r) -> Row {
    r = min(r, rows - 1);
    const int k = by_rows(r), h = r - k * all, token = token0 + k, b = by_nodes(token);
    const bool key = h >= a.q.heads;
    return {key ? &a.k : &a.q, k, b, token - b * a.nodes, key ? h - a.q.heads : h};
  };
  auto load = [&](const Row& r, uint4 (&raw)[2]) {
    const T* from = static_cast<const T*>(r.kind->x) + r.b * r.kind->x_seq + r.node * r.kind->x_node +
                    r.head * r.kind->x_head + e;
    raw[0] = *reinterpret_cast<const uint4*>(from);
    raw[1] = *reinterpret_cast<const uint4*>(from + kHalf);
  };
  const int first = split * kRows, step = splits * kRows, mine = threadIdx.x / kLanes;
  Row next_row = row_of(first + mine);
  uint4 next[2];
  load(next_row, next);
  for (int i = threadIdx.x; i < here * half; i += kThreads) {
    const int k = i / half, token = token0 + k, b = by_nodes(token);
    const int pos = a.positions[b * a.stride_positions + token - b * a.nodes];
    // The angle in turns; whole turns are dropped in fp64.
    const double t = pos * a.inv_freq[i - k * half] * kTurn;
    float s, c;
    sincospif(static_cast<float>(2.0 * (t - rint(t))), &s, &c);
    cosines[i] = c;
    sines[i] = s;
  }
  if (threadIdx.x < here) {
    const int token = token0 + threadIdx.x, b = by_nodes(token);
    positions[threadIdx.x] = a.positions[b * a.stride_positions + token - b * a.nodes];
  }
  __syncthreads();
  const bool interleaved = a.flags & TF_QK_INTERLEAVED, hadamard = a.flags & TF_QK_HADAMARD;
  // Whole warps run through the loop together, so that lanes can meet.
#pragma unroll 1
  for (int r0 = first; r0 < rows; r0 += step) {
    const Row row = next_row;
    // x[0][..] are elements e .. e + 7, x[1][..] those half a head on.
    float2 x[2][4], w[2][4];
    pairs_of<T>(next[0], x[0]);
    pairs_of<T>(next[1], x[1]);
    if (r0 + step < rows) {
      next_row = row_of(r0 + step + mine);
      load(next_row, next);
    }
    load_weight<W>(row.kind->weight, e, w[0]);
    load_weight<W>(row.kind->weight, e + kHalf, w[1]);
    float f = 1.f;
    if (!(a.flags & TF_QK_NO_NORM)) {
      auto mean_square = [&]() {
        float2 both = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) both = fma2(x[i / 4][i % 4], x[i / 4][i % 4], both);
        float sum = both.x + both.y;
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
        return sum * (1.f / D);
      };
      float square = mean_square() + a.eps;
      // Squares of large or small bf16 numbers pass fp32's range where the
      // numbers don't: such rows are scaled by a power of two first (2^-70: the
      // sum of 256 squares is below 2^128, and what is left of the row as a bf16
      // number, 2^-126 of its root mean square and more, keeps 8 bits).
      if (std::is_same<T, __nv_bfloat16>::value &&
          __any_sync(~0u, square >= 0x1p120f || square < 0x1p-80f)) {
        const float by = square >= 0x1p120f ? 0x1p-70f : square < 0x1p-80f ? 0x1p90f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i / 4][i % 4] = mul2(x[i / 4][i % 4], twice(by));
        square = mean_square() + a.eps * by * by;
      }
      f = rsqrtf(square);
    }
    if (hadamard) f *= D == 64 ? 0.125f : D == 128 ? 0.0883883476f : 0.0625f;   // 1 / sqrt(D)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i / 4][i % 4] = mul2(mul2(x[i / 4][i % 4], twice(f)), w[i / 4][i % 4]);
    const float* cs = cosines + row.k * half;
    const float* sn = sines + row.k * half;
    if (half > 0 && interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = e + i / 4 * kHalf + i % 4 * 2;
        if (d < a.rotary) {
          const float2 v = x[i / 4][i % 4];
          const float c = cs[d / 2], s = sn[d / 2];
          x[i / 4][i % 4] = float2{v.x * c - v.y * s, v.y * c + v.x * s};
        }
      }
    } else if (a.rotary == D) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = *reinterpret_cast<const float2*>(cs + e + 2 * i);
        const float2 s = *reinterpret_cast<const float2*>(sn + e + 2 * i);
        const float2 u = x[0][i], v = x[1][i];
        x[0][i] = minus(mul2(u, c), mul2(v, s));
        x[1][i] = fma2(v, c, mul2(u, s));
      }
    } else if (half > 0) {
      // The pairs of a piece of 8 elements lie half / 8 pieces away, in either
      // half of another lane.
      float2 y[2][4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int piece = lane + p * kLanes, d = piece * 8;
        const bool turned = d < a.rotary, low = d < half;
        const int other = !turned ? piece : low ? piece + half / 8 : piece - half / 8;
        const int from = static_cast<int>(threadIdx.x % 32) - lane + other % kLanes;
        const int at = turned ? (low ? d : d - half) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 z[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            z[k] = float2{__shfl_sync(~0u, x[k][i].x, from), __shfl_sync(~0u, x[k][i].y, from)};
          const float2 v = other < kLanes ? z[0] : z[1];
          const float2 c = *reinterpret_cast<const float2*>(cs + at + 2 * i);
          const float2 s = *reinterpret_cast<const float2*>(sn + at + 2 * i);
          y[p][i] = x[p][i];
          if (turned) y[p][i] = fma2(mul2(v, s), twice(low ? -1.f : 1.f), mul2(x[p][i], c));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i / 4][i % 4] = y[i / 4][i % 4];
    }
    if (hadamard) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // neighbours
        const float2 v = x[i / 4][i % 4];
        x[i / 4][i % 4] = float2{v.x + v.y, v.x - v.y};
      }
#pragma unroll
      for (int o = 1; o < 8; o *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & o)) {
            const int j = i + o;
            const float2 u = x[i / 4][i % 4], v = x[j / 4][j % 4];
            x[i / 4][i % 4] = add2(u, v);
            x[j / 4][j % 4] = minus(u, v);
          }
#pragma unroll
      for (int o = 1; o < kLanes; o *= 2) {
        const float2 sign = twice(lane & o ? -1.f : 1.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = x[i / 4][i % 4];
          x[i / 4][i % 4] = fma2(v, sign, float2{__shfl_xor_sync(~0u, v.x, o), __shfl_xor_sync(~0u, v.y, o)});
        }
      }
    }
    if (r0 + mine < rows && positions[row.k] >= 0) {
      T* to = static_cast<T*>(row.kind->y) + row.b * row.kind->y_seq + row.node * row.kind->y_node +
              row.head * row.kind->y_head + e;
      *reinterpret_cast<uint4*>(to) = pack8<T>(*reinterpret_cast<const float(*)[8]>(x[0]));
      *reinterpret_cast<uint4*>(to + kHalf) = pack8<T>(*reinterpret_cast<const float(*)[8]>(x[1]));
    }
  }
}

template <typename T, typename W>
cudaError_t launch(const NormRopeArgs& a, int head_dim, cudaStream_t s) {
  const int rows = kThreads / (head_dim / 16), all = a.q.heads + a.k.heads, tokens = a.batch * a.nodes;
  // Few tokens: a block for each `rows` heads of one. Many: as many tokens a
  // block as its threads can have the angles of, but every SM some blocks.
  const int splits = tokens < 4 * a.num_sms ? (all + rows - 1) / rows : 1;
  const int per_block = std::max(1, std::min(kThreads / std::max(a.rotary / 2, 32), tokens / (8 * a.num_sms)));
  const dim3 grid(static_cast<unsigned>((tokens + per_block - 1) / per_block * splits));
  const FastDiv by_nodes(static_cast<uint32_t>(a.nodes)), by_rows(static_cast<uint32_t>(all));
  auto with = [&](auto kernel) {
    return launch_chained(kernel, grid, dim3(kThreads), 0, 1, s, a, tokens, per_block, splits, by_nodes, by_rows);
  };
  switch (head_dim) {
    case 64: return with(qk_norm_rope_kernel<T, W, 64>);
    case 128: return with(qk_norm_rope_kernel<T, W, 128>);
    default: return with(qk_norm_rope_kernel<T, W, 256>);
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
