// Rows of the quantised cache: written (tf_kvq_write), read back
// (tf_kvq_read), moved (tf_kvq_keep).
//
// head_dim / 8 lanes have a token's or slot's rows of kAtOnce heads, 8 elements
// of a row each, keys and values side by side, so that one lane writes both
// factors as one word. A page is looked up once for those heads (a look-up for
// each row was most of the instructions: a batch of 16 contexts of up to 4,096
// slots read in 66 us), and their rows are in flight together. What bounds
// them is the launch for a few tokens and for many memory (reading) or
// instructions (writing: conversions, maxima, codes).
// Measured, 8 heads of 128: 16 parts of 512 tokens written in 8 bits 15.8 us
// (50 MB, issue slots 62% busy), with their reading back 22.5; 16 contexts of
// up to 4,096 slots read from 4 bits into 16 in 37.6 (211 MB, 5.6 TB/s); the
// paths of 32 sequences kept in 32 layers in 9.3 (21 MB).
#include <algorithm>
#include <type_traits>

#include "qcache.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 256;

// Codes of eight elements of a row whose largest magnitude is `top` (finite),
// and the row's factor. The definition is round(x / s), to the nearest, ties to
// even. x has at most 11 significant bits and s 8, so that a quotient below 128
// that is no tie is at least 2^-12 from one; x times 1 / s, which may be off by
// a unit in its last place, is off by 2^-15 at most. Rounding it to a multiple
// of 2^-13 first (the addition of 1.5 * 2^10) makes a tie exact and moves
// nothing else across one, in two additions instead of a division. s is off
// by 2^-9 of itself at most, so that no quotient rounds to more than 7 or 127.
// Rows whose factor is not in the middle of fp32's range are divided.
template <int kBits>
__device__ __noinline__ uint64_t quantise8_by_division(float4 a, float4 b, float s) {
  constexpr float kMost = kBits == 4 ? 7.f : 127.f;
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint64_t out = 0;
#pragma unroll 1
  for (int i = 7; i >= 0; --i)
    out = out << kBits | static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(__fdiv_rn(x[i], s), -kMost), kMost)) +
                                               (1 << (kBits - 1)));
  return out;
}
// bf16(top / m) in every bit: the quotient of a number by a small constant is
// its product with the rounded reciprocal, corrected once by what is left
// (Markstein, Computation of elementary functions on the IBM RISC System/6000).
template <int kBits>
__device__ __noinline__ float factor_by_division(float top) {
  return __bfloat162float(__float2bfloat16_rn(__fdiv_rn(top, kBits == 4 ? 7.f : 127.f)));
}
template <int kBits>
__device__ __forceinline__ float factor_of(float top) {
  constexpr float kMost = kBits == 4 ? 7.f : 127.f, kInv = 1.f / kMost;
  if (top < 0x1p-90f || top > 0x1p90f) return factor_by_division<kBits>(top);
  const float q = __fmul_rn(top, kInv), s = __fmaf_rn(__fmaf_rn(-kMost, q, top), kInv, q);
  return __bfloat162float(__float2bfloat16_rn(s));
}
// Whole numbers below 2^22 as the lowest bits of their fp32 sum with this.
constexpr float kWhole = 12582912.f;   // 1.5 * 2^23

template <int kBits>
__device__ __forceinline__ uint64_t quantise8(const float (&x)[8], float s) {
  if (s == 0.f) return kBits == 4 ? 0x88888888ull : 0x8080808080808080ull;
  if (s < 0x1p-100f || s > 0x1p100f)
    return quantise8_by_division<kBits>(float4{x[0], x[1], x[2], x[3]}, float4{x[4], x[5], x[6], x[7]}, s);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  float2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // two whole numbers each
    t[i] = mul2(float2{x[2 * i], x[2 * i + 1]}, float2{inv, inv});
    t[i] = add2(add2(t[i], float2{1536.f, 1536.f}), float2{-1536.f, -1536.f});
    t[i] = add2(add2(t[i], float2{kWhole, kWhole}), float2{-kWhole, -kWhole});
  }
  // Several of them as one whole number of 16 bits, exactly, with the bias.
  uint32_t w[4];
  if (kBits == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = __fmaf_rn(16.f, t[2 * i].y, t[2 * i].x), b = __fmaf_rn(16.f, t[2 * i + 1].y, t[2 * i + 1].x);
      w[i] = __float_as_uint(__fmaf_rn(256.f, b, a) + (kWhole + 0x8888));
    }
    return __byte_perm(w[0], w[1], 0x5410);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__fmaf_rn(256.f, t[i].y, t[i].x) + (kWhole + 0x8080));
  return __byte_perm(w[0], w[1], 0x5410) | static_cast<uint64_t>(__byte_perm(w[2], w[3], 0x5410)) << 32;
}

// The largest magnitude of a row of 16-bit elements, as the element's bits
// (which order magnitudes, infinity and NaN last), for all its lanes.
template <int kLanes>
__device__ __forceinline__ uint32_t row_top(const uint4& w) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t top = __vmaxu2(__vmaxu2(w.x & kAbs, w.y & kAbs), __vmaxu2(w.z & kAbs, w.w & kAbs));
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
  return max(top & 0xFFFFu, top >> 16);
}

// Eight elements of a row: codes, and the factor's bits.
template <typename T, int kBits, int kLanes>
__device__ __forceinline__ uint64_t quantise(const uint4& w, uint16_t* factor) {
  constexpr uint32_t kInfinity = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  const uint32_t bits = row_top<kLanes>(w);
  if (bits >= kInfinity) {   // a row that is not finite
    *factor = 0x7FC0;
    return kBits == 4 ? 0x88888888ull : 0x8080808080808080ull;
  }
  const uint16_t b16 = static_cast<uint16_t>(bits);
  const float s = factor_of<kBits>(to_f32(*reinterpret_cast<const T*>(&b16)));
  float x[8];
  unpack8<T>(w, x);
  *factor = static_cast<uint16_t>(__float_as_uint(s) >> 16);
  return quantise8<kBits>(x, s);
}

constexpr int kAtOnce = 4;

// The units of a call: kAtOnce heads of one of a sequence's `tokens` tokens.
struct Units {
  uint32_t count;   // below 2^31, so that a step past the end does not wrap
  int chunks;
  FastDiv by_chunks, by_tokens;
  Units(int batch, int tokens, int heads)
      : chunks((heads + kAtOnce - 1) / kAtOnce), by_chunks(static_cast<uint32_t>(chunks)),
        by_tokens(static_cast<uint32_t>(tokens)) {
    count = static_cast<uint32_t>(batch) * tokens * chunks;
  }
};

// Whole warps run through the loops together, so that a row's lanes can meet.
template <typename T, int kBits, int D>
__global__ void __launch_bounds__(kThreads)
kvq_write_kernel(const __grid_constant__ QView q, const __grid_constant__ RowsIn k_new,
                 const __grid_constant__ RowsIn v_new, const int32_t* counts, int nodes, Units units) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  chain();
  const int lane = threadIdx.x % kLanes;
  for (uint32_t u0 = blockIdx.x * kGroups; u0 < units.count; u0 += gridDim.x * kGroups) {
    const uint32_t unit = u0 + threadIdx.x / kLanes;
    const bool in = unit < units.count;
    const int token = in ? units.by_chunks(unit) : 0, h0 = in ? (unit - token * units.chunks) * kAtOnce : 0;
    const int b = units.by_tokens(token), i = token - b * nodes;
    const T* k_row = static_cast<const T*>(k_new.at) + b * k_new.seq + i * k_new.node + lane * 8;
    const T* v_row = static_cast<const T*>(v_new.at) + b * v_new.seq + i * v_new.node + lane * 8;
    int n = counts ? counts[b] : nodes;
    if (n < 0 || n > nodes) {
      if (in) record_index_error(q.c.err);
      n = n < 0 ? 0 : nodes;
    }
    uint4 kw[kAtOnce], vw[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      kw[u] = vw[u] = uint4{0, 0, 0, 0};
      if (in && i < n && h0 + u < q.c.kv_heads) {
        kw[u] = *reinterpret_cast<const uint4*>(k_row + (h0 + u) * k_new.head);
        vw[u] = *reinterpret_cast<const uint4*>(v_row + (h0 + u) * v_new.head);
      }
    }
    const int len = q.c.lengths[b];
    Place at = {0, 0};
    const bool real = in && len >= 0 && i < n && place_of(q.c, b, static_cast<int64_t>(len) + i, &at);
    uint8_t* k_to = q.k + codes_at(q.c, at) + lane * kBits;
    uint8_t* v_to = q.v + codes_at(q.c, at) + lane * kBits;
    uint32_t* s_to = q.scales + scales_at(q, at);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      uint16_t ks, vs;
      const uint64_t kc = quantise<T, kBits, kLanes>(kw[u], &ks), vc = quantise<T, kBits, kLanes>(vw[u], &vs);
      if (!real || h0 + u >= q.c.kv_heads) continue;
      const int64_t dst = (h0 + u) * q.c.stride_head;
      if (kBits == 4) {
        *reinterpret_cast<uint32_t*>(k_to + dst) = static_cast<uint32_t>(kc);
        *reinterpret_cast<uint32_t*>(v_to + dst) = static_cast<uint32_t>(vc);
      } else {
        *reinterpret_cast<uint64_t*>(k_to + dst) = kc;
        *reinterpret_cast<uint64_t*>(v_to + dst) = vc;
      }
      if (lane == 0) s_to[(h0 + u) * q.scale_head] = ks | static_cast<uint32_t>(vs) << 16;
    }
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
                int64_t head, int slots, Units units) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  chain();
  const int lane = threadIdx.x % kLanes;
  for (uint32_t unit = blockIdx.x * kGroups + threadIdx.x / kLanes; unit < units.count; unit += gridDim.x * kGroups) {
    const int id = units.by_chunks(unit), h0 = (unit - id * units.chunks) * kAtOnce;
    const int b = units.by_tokens(id), i = id - b * slots;
    const int start = starts ? starts[b] : 0;
    if (start < 0) {
      record_index_error(q.c.err);
      continue;
    }
    const int64_t s = static_cast<int64_t>(start) + i;
    Place at;
    if (s >= q.c.lengths[b] || !place_of(q.c, b, s, &at)) continue;
    const uint8_t* k_from = q.k + codes_at(q.c, at) + lane * kBits;
    const uint8_t* v_from = q.v + codes_at(q.c, at) + lane * kBits;
    const uint32_t* s_from = q.scales + scales_at(q, at);
    T* k_to = k_out + b * seq + i * slot + lane * 8;
    T* v_to = v_out + b * seq + i * slot + lane * 8;
    uint64_t kc[kAtOnce], vc[kAtOnce];
    uint32_t w[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (h0 + u >= q.c.kv_heads) break;
      const int64_t src = (h0 + u) * q.c.stride_head;
      w[u] = s_from[(h0 + u) * q.scale_head];
      if (kBits == 4) {
        kc[u] = *reinterpret_cast<const uint32_t*>(k_from + src);
        vc[u] = *reinterpret_cast<const uint32_t*>(v_from + src);
      } else {
        kc[u] = *reinterpret_cast<const uint64_t*>(k_from + src);
        vc[u] = *reinterpret_cast<const uint64_t*>(v_from + src);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (h0 + u >= q.c.kv_heads) break;
      *reinterpret_cast<uint4*>(k_to + (h0 + u) * head) = values8<T, kBits>(kc[u], key_scale(w[u]));
      *reinterpret_cast<uint4*>(v_to + (h0 + u) * head) = values8<T, kBits>(vc[u], value_scale(w[u]));
    }
  }
}

constexpr int kAhead = 8;

template <typename W, typename From, typename To>
__device__ __forceinline__ void move_along(int n, const Place* from, From&& source, To&& target) {
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    W w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u < n && from[i0 + u].page >= 0) w[u] = *source(i0 + u);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u < n && from[i0 + u].page >= 0) *target(i0 + u) = w[u];
  }
}

// A block moves the codes and factors of one sequence and layer; a thread one
// 16-byte chunk of codes, or one word of factors, along the whole path. The
// path rises: entry k goes from slot path[k] >= k to slot k, so that no later
// source is written by an earlier move, and kAhead moves are loaded before
// the first of them is stored (32 paths of 16 in 32 layers, 8 bits, 9.4 us one
// by one).
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
  int n = counts[b];
  if (n < 0 || n > nodes) {
    if (threadIdx.x == 0) record_index_error(q.c.err);
    n = n < 0 ? 0 : nodes;
  }
  if (threadIdx.x == 0) kept = n;
  __syncthreads();
  const int entry = threadIdx.x, p = entry < n ? path[b * nodes + entry] : 0;
  if (entry < n && (p >= nodes || p <= (entry ? path[b * nodes + entry - 1] : -1))) {
    record_index_error(q.c.err);
    atomicMin(&kept, entry);   // the path is followed up to here
  }
  __syncthreads();
  n = kept;
  if (blockIdx.x == 0 && layer == 0 && entry == 0) new_lengths[b] = len + n;
  if (entry < n) {
    Place x = {-1, 0}, y = {-1, 0};
    if (p == entry || !place_of(q.c, b, static_cast<int64_t>(len) + p, &x) ||
        !place_of(q.c, b, static_cast<int64_t>(len) + entry, &y))
      x.page = -1;
    from[entry] = x;
    to[entry] = y;
  }
  __syncthreads();
  const int chunks = q.c.head_dim * q.bits / 128, units = q.c.kv_heads * (2 * chunks + 1);
  for (int id = blockIdx.x * kThreads + threadIdx.x; id < units; id += gridDim.x * kThreads) {
    const int h = id / (2 * chunks + 1), rest = id - h * (2 * chunks + 1);
    if (rest < 2 * chunks) {
      uint8_t* base = (rest < chunks ? q.k : q.v) + layer * q.c.stride_layer + h * q.c.stride_head +
                      (rest < chunks ? rest : rest - chunks) * 16;
      move_along<uint4>(n, from, [&](int i) { return reinterpret_cast<uint4*>(base + codes_at(q.c, from[i])); },
                        [&](int i) { return reinterpret_cast<uint4*>(base + codes_at(q.c, to[i])); });
    } else {
      uint32_t* base = q.scales + layer * q.scale_layer + h * q.scale_head;
      move_along<uint32_t>(n, from, [&](int i) { return base + scales_at(q, from[i]); },
                           [&](int i) { return base + scales_at(q, to[i]); });
    }
  }
}

// One launch of a kernel that goes through the units.
template <typename... P, typename... A>
cudaError_t launch_units(void (*kernel)(P...), const Units& units, int head_dim, cudaStream_t s, A&&... args) {
  const int per = kThreads / (head_dim / 8), blocks = static_cast<int>((units.count - 1) / per) + 1;
  return launch_chained(kernel, dim3(std::min(blocks, 32768)), dim3(kThreads), 0, 1, s, static_cast<A&&>(args)..., units);
}

template <typename T, int kBits, int D>
struct Kernels {
  static cudaError_t write(const QView& q, const RowsIn& k, const RowsIn& v, const int32_t* counts, int nodes,
                           cudaStream_t s) {
    return launch_units(kvq_write_kernel<T, kBits, D>, Units(q.c.batch, nodes, q.c.kv_heads), D, s, q, k, v, counts,
                        nodes);
  }
  static cudaError_t read(const QView& q, const int32_t* starts, void* k, void* v, int64_t seq, int64_t slot,
                          int64_t head, int slots, cudaStream_t s) {
    return launch_units(kvq_read_kernel<T, kBits, D>, Units(q.c.batch, slots, q.c.kv_heads), D, s, q, starts,
                        static_cast<T*>(k), static_cast<T*>(v), seq, slot, head, slots);
  }
};

// f(Kernels<...>()) of the call's type, width and head size.
template <typename T, int kBits, typename F>
cudaError_t by_dim(int head_dim, F&& f) {
  return head_dim == 64    ? f(Kernels<T, kBits, 64>())
         : head_dim == 128 ? f(Kernels<T, kBits, 128>())
                           : f(Kernels<T, kBits, 256>());
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
