// Rows of the quantised cache: written (tf_kvq_write), read back
// (tf_kvq_read), moved (tf_kvq_keep). head_dim / 8 lanes have a row of one
// head, 8 elements each, keys and values side by side, so that one lane writes
// both factors as one word. What bounds them is the launch for a few tokens
// and memory for many.
#include "qcache.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 256;

// Codes of eight elements of a row whose largest magnitude has the bits `top`
// (as fp32), and the row's factor. The definition is round(x / s), to the
// nearest, ties to even. x has at most 11 significant bits and s 8, so that a
// quotient below 128 that is no tie is at least 2^-12 from one; x times the
// rounded 1 / s is off by 2^-16 at most. Rounding it to a multiple of 2^-13
// first (the addition of 1.5 * 2^10) makes a tie exact and moves nothing else
// across one, in two additions instead of a division. Factors whose
// reciprocal leaves fp32's normal range are divided by.
template <int kBits>
__device__ __forceinline__ uint64_t quantise8(const float (&x)[8], uint32_t top, uint16_t* factor) {
  constexpr float kMost = kBits == 4 ? 7.f : 127.f;
  constexpr int kBias = kBits == 4 ? 8 : 128;
  uint64_t out = 0;
  const bool finite = top < 0x7F800000u;
  const __nv_bfloat16 s16 = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), kMost));
  const float s = __bfloat162float(s16);
  *factor = finite ? __bfloat16_as_ushort(s16) : static_cast<uint16_t>(0x7FC0);
  const bool none = !finite || s == 0.f, plain = s >= 0x1p-100f && s <= 0x1p100f;
  const float inv = __fdiv_rn(1.f, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = plain ? __fadd_rn(__fadd_rn(__fmul_rn(x[i], inv), 1536.f), -1536.f) : __fdiv_rn(x[i], s);
    const int c = none ? 0 : __float2int_rn(fminf(fmaxf(t, -kMost), kMost));
    out |= static_cast<uint64_t>(static_cast<uint32_t>(c + kBias)) << (i * kBits);
  }
  return out;
}

template <int kLanes>
__device__ __forceinline__ uint32_t row_top(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) top = max(top, __shfl_xor_sync(~0u, top, o));
  return top;
}

// Whole warps run through the loop together, so that the rows' lanes can meet.
template <typename T, int kBits, int D>
__global__ void __launch_bounds__(kThreads)
kvq_write_kernel(const __grid_constant__ QView q, const __grid_constant__ RowsIn k_new,
                 const __grid_constant__ RowsIn v_new, const int32_t* counts, int nodes) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  chain();
  const int lane = threadIdx.x % kLanes;
  const int64_t rows = static_cast<int64_t>(q.c.batch) * nodes * q.c.kv_heads;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t id = r0 + threadIdx.x / kLanes;
    const int64_t token = id / q.c.kv_heads;
    const int h = static_cast<int>(id - token * q.c.kv_heads);
    const int b = static_cast<int>(token / nodes), i = static_cast<int>(token - static_cast<int64_t>(b) * nodes);
    bool real = id < rows;
    Place at = {0, 0};
    if (real) {
      const int len = q.c.lengths[b];
      int n = counts ? counts[b] : nodes;
      if (n < 0 || n > nodes) {
        record_index_error(q.c.err);
        n = n < 0 ? 0 : nodes;
      }
      real = len >= 0 && i < n && place_of(q.c, b, static_cast<int64_t>(len) + i, &at);
    }
    auto row = [&](const RowsIn& r) {
      return *reinterpret_cast<const uint4*>(static_cast<const T*>(r.at) + b * r.seq + i * r.node + h * r.head + lane * 8);
    };
    float x[8] = {}, y[8] = {};
    if (real) {
      unpack8<T>(row(k_new), x);
      unpack8<T>(row(v_new), y);
    }
    uint16_t ks, vs;
    const uint64_t kc = quantise8<kBits>(x, row_top<kLanes>(x), &ks);
    const uint64_t vc = quantise8<kBits>(y, row_top<kLanes>(y), &vs);
    if (!real) continue;
    const int64_t dst = codes_at(q.c, at) + h * q.c.stride_head + lane * kBits;
    if (kBits == 4) {
      *reinterpret_cast<uint32_t*>(q.k + dst) = static_cast<uint32_t>(kc);
      *reinterpret_cast<uint32_t*>(q.v + dst) = static_cast<uint32_t>(vc);
    } else {
      *reinterpret_cast<uint64_t*>(q.k + dst) = kc;
      *reinterpret_cast<uint64_t*>(q.v + dst) = vc;
    }
    if (lane == 0) q.scales[scales_at(q, at) + h * q.scale_head] = ks | static_cast<uint32_t>(vs) << 16;
  }
}

template <typename T, int kBits>
__device__ __forceinline__ uint4 values8(uint64_t codes, float s) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = (static_cast<int>(codes >> (i * kBits) & ((1u << kBits) - 1)) - (1 << (kBits - 1))) * s;
  return pack8<T>(x);
}

template <typename T, int kBits, int D>
__global__ void __launch_bounds__(kThreads)
kvq_read_kernel(const __grid_constant__ QView q, const int32_t* starts, T* k_out, T* v_out, int64_t seq, int64_t slot,
                int64_t head, int slots) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  chain();
  const int lane = threadIdx.x % kLanes;
  const int64_t rows = static_cast<int64_t>(q.c.batch) * slots * q.c.kv_heads;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kLanes; id < rows;
       id += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t token = id / q.c.kv_heads;
    const int h = static_cast<int>(id - token * q.c.kv_heads);
    const int b = static_cast<int>(token / slots), i = static_cast<int>(token - static_cast<int64_t>(b) * slots);
    const int start = starts ? starts[b] : 0;
    if (start < 0) {
      record_index_error(q.c.err);
      continue;
    }
    const int64_t s = static_cast<int64_t>(start) + i;
    Place at;
    if (s >= q.c.lengths[b] || !place_of(q.c, b, s, &at)) continue;
    const int64_t src = codes_at(q.c, at) + h * q.c.stride_head + lane * kBits;
    const uint32_t w = q.scales[scales_at(q, at) + h * q.scale_head];
    uint64_t kc, vc;
    if (kBits == 4) {
      kc = *reinterpret_cast<const uint32_t*>(q.k + src);
      vc = *reinterpret_cast<const uint32_t*>(q.v + src);
    } else {
      kc = *reinterpret_cast<const uint64_t*>(q.k + src);
      vc = *reinterpret_cast<const uint64_t*>(q.v + src);
    }
    const int64_t dst = b * seq + i * slot + h * head + lane * 8;
    *reinterpret_cast<uint4*>(k_out + dst) = values8<T, kBits>(kc, key_scale(w));
    *reinterpret_cast<uint4*>(v_out + dst) = values8<T, kBits>(vc, value_scale(w));
  }
}

// A block moves the codes and factors of one sequence and layer; a thread one
// 16-byte chunk of codes, or one word of factors, along the whole path. The
// path rises: entry k goes from slot path[k] >= k to slot k, so that no later
// source is written by an earlier move, and kAhead moves are loaded before
// the first of them is stored.
__global__ void __launch_bounds__(kThreads)
kvq_keep_kernel(const __grid_constant__ QView q, const int32_t* path, const int32_t* counts, int nodes,
                int32_t* new_lengths) {
  __shared__ Place from[TF_MAX_NODES], to[TF_MAX_NODES];
  __shared__ int kept;
  chain();
  const int b = blockIdx.y, layer = blockIdx.z;
  const int len = q.c.lengths[b];
  if (len < 0) {
    if (blockIdx.x == 0 && layer == 0 && threadIdx.x == 0) new_lengths[b] = len;
    return;
  }
  if (threadIdx.x == 0) {
    int n = counts[b];
    if (n < 0 || n > nodes) {
      record_index_error(q.c.err);
      n = n < 0 ? 0 : nodes;
    }
    int last = -1, i = 0;
    for (; i < n; ++i) {
      const int p = path[b * nodes + i];
      if (p <= last || p >= nodes) {
        record_index_error(q.c.err);
        break;
      }
      last = p;
    }
    kept = i;
    if (blockIdx.x == 0 && layer == 0) new_lengths[b] = len + i;
  }
  __syncthreads();
  const int n = kept;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int p = path[b * nodes + i];
    Place x = {-1, 0}, y = {-1, 0};
    if (p == i || !place_of(q.c, b, static_cast<int64_t>(len) + p, &x) ||
        !place_of(q.c, b, static_cast<int64_t>(len) + i, &y))
      x.page = -1;
    from[i] = x;
    to[i] = y;
  }
  __syncthreads();
  const int chunks = q.c.head_dim * q.bits / 128, units = q.c.kv_heads * (2 * chunks + 1);
  for (int id = blockIdx.x * kThreads + threadIdx.x; id < units; id += gridDim.x * kThreads) {
    const int h = id / (2 * chunks + 1), rest = id - h * (2 * chunks + 1);
    if (rest < 2 * chunks) {
      uint8_t* base = (rest < chunks ? q.k : q.v) + layer * q.c.stride_layer + h * q.c.stride_head +
                      (rest < chunks ? rest : rest - chunks) * 16;
      for (int i = 0; i < n; ++i)
        if (from[i].page >= 0)
          *reinterpret_cast<uint4*>(base + codes_at(q.c, to[i])) =
              *reinterpret_cast<const uint4*>(base + codes_at(q.c, from[i]));
    } else {
      uint32_t* base = q.scales + layer * q.scale_layer + h * q.scale_head;
      for (int i = 0; i < n; ++i)
        if (from[i].page >= 0) base[scales_at(q, to[i])] = base[scales_at(q, from[i])];
    }
  }
}

// One launch of a kernel that goes through `rows` rows.
template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), int64_t rows, int head_dim, cudaStream_t s, A&&... args) {
  const int64_t per = kThreads / (head_dim / 8), blocks = (rows + per - 1) / per;
  return launch_chained(kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0, 1, s,
                        static_cast<A&&>(args)...);
}

template <typename T, int kBits, int D>
struct Kernels {
  static cudaError_t write(const QView& q, const RowsIn& k, const RowsIn& v, const int32_t* counts, int nodes,
                           cudaStream_t s) {
    return launch_rows(kvq_write_kernel<T, kBits, D>, static_cast<int64_t>(q.c.batch) * nodes * q.c.kv_heads, D, s, q, k,
                       v, counts, nodes);
  }
  static cudaError_t read(const QView& q, const int32_t* starts, void* k, void* v, int64_t seq, int64_t slot,
                          int64_t head, int slots, cudaStream_t s) {
    return launch_rows(kvq_read_kernel<T, kBits, D>, static_cast<int64_t>(q.c.batch) * slots * q.c.kv_heads, D, s, q,
                       starts, static_cast<T*>(k), static_cast<T*>(v), seq, slot, head, slots);
  }
};

// f(Kernels<...>()) of the call's type, width and head size.
template <typename T, int kBits, typename F>
cudaError_t by_dim(int head_dim, F&& f) {
  return head_dim == 64 ? f(Kernels<T, kBits, 64>()) : head_dim == 128 ? f(Kernels<T, kBits, 128>()) : f(Kernels<T, kBits, 256>());
}
template <typename F>
cudaError_t by_kind(int dtype, int bits, int head_dim, F&& f) {
  if (dtype == TF_F16) return bits == 4 ? by_dim<__half, 4>(head_dim, f) : by_dim<__half, 8>(head_dim, f);
  return bits == 4 ? by_dim<__nv_bfloat16, 4>(head_dim, f) : by_dim<__nv_bfloat16, 8>(head_dim, f);
}

}  // namespace

cudaError_t launch_kvq_write(const QView& q, const RowsIn& k_new, const RowsIn& v_new, int dtype,
                             const int32_t* counts, int nodes, cudaStream_t s) {
  return by_kind(dtype, q.bits, q.c.head_dim,
                 [&](auto kernels) { return kernels.write(q, k_new, v_new, counts, nodes, s); });
}

cudaError_t launch_kvq_read(const QView& q, const int32_t* starts, void* k_out, void* v_out, int dtype, int64_t seq,
                            int64_t slot, int64_t head, int slots, cudaStream_t s) {
  return by_kind(dtype, q.bits, q.c.head_dim, [&](auto kernels) {
    return kernels.read(q, starts, k_out, v_out, seq, slot, head, slots, s);
  });
}

cudaError_t launch_kvq_keep(const QView& q, const int32_t* path, const int32_t* counts, int nodes,
                            int32_t* new_lengths, cudaStream_t s) {
  const int units = q.c.kv_heads * (q.c.head_dim * q.bits / 64 + 1);
  return launch_chained(kvq_keep_kernel, dim3((units + kThreads - 1) / kThreads, q.c.batch, q.c.layers), dim3(kThreads), 0,
                        1, s, q, path, counts, nodes, new_lengths);
}

}  // namespace tfx
