// Device helpers shared by the cache, attention and verification kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "spec.h"

namespace tfx {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// In every thread of a kernel launched by launch_chained: waits for the kernel
// before it, and lets the next one be set up.
__device__ __forceinline__ void chain() {
  pdl_wait_prerequisites();
  pdl_launch_dependents();
}

// The two halves of a barrier over all threads of a cluster.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ void record_index_error(int* err) { atomicOr(err, kErrIndex); }

// Slots a sequence's page table can name (below 2^31 by the host's check).
__device__ __forceinline__ int slot_capacity(const CacheView& c) { return c.table_width * c.page_size; }

// What exists of a sequence: its context slots and the slots up to its last
// node. A length the table cannot hold is cut to what it can (recorded).
struct Span {
  int context, slots;  // -1, 0 for an idle sequence
};
__device__ __forceinline__ Span sequence_span(const CacheView& c, int b, int nodes) {
  const int len = __ldcg(c.lengths + b), cap = slot_capacity(c);
  if (len < 0) return {-1, 0};
  if (len <= cap - nodes) return {len, len + nodes};
  record_index_error(c.err);
  return {min(len, cap), cap};
}

// Offset of slot `slot` of sequence `b` (layer 0, head 0), or -1 where the
// slot lies past the table or its page outside the pool (recorded).
__device__ __forceinline__ int64_t slot_offset(const CacheView& c, int b, int64_t slot) {
  if (slot < 0 || slot >= slot_capacity(c)) {
    record_index_error(c.err);
    return -1;
  }
  const int p = c.by_page(static_cast<int>(slot));
  const int page = c.page_table[b * c.stride_table + p];
  if (page < 0 || page >= c.pages) {
    record_index_error(c.err);
    return -1;
  }
  return page * c.stride_page + (static_cast<int>(slot) - p * c.page_size) * c.stride_token;
}

// The ancestors of up to kNodes nodes as bit masks: sees(i, j) when row i sees
// node j (itself or an ancestor, none absent). Built in log2(nodes) rounds of
// pointer doubling, by all threads of a block of at least kNodes.
template <int kNodes>
struct TreeMasks {
  static constexpr int kWords = (kNodes + 31) / 32;
  uint32_t anc[kNodes][kWords];
  int16_t up[kNodes];

  __device__ __forceinline__ bool sees(int i, int j) const { return anc[i][j >> 5] >> (j & 31) & 1; }

  __device__ __forceinline__ void build(const int32_t* parents, int nodes, int* err) {
    const int j = threadIdx.x;
    if (j < nodes) {
      int p = parents[j];
      if (p >= j) {
        record_index_error(err);
        p = -2;
      }
      for (int w = 0; w < kWords; ++w) anc[j][w] = 0;
      if (p >= -1) anc[j][j >> 5] = 1u << (j & 31);
      up[j] = p >= 0 ? p : -1;
    }
    __syncthreads();
    for (int span = 1; span < nodes; span *= 2) {
      uint32_t m[kWords] = {};
      int next = -1;
      if (j < nodes && up[j] >= 0) {
        const int p = up[j];
        for (int w = 0; w < kWords; ++w) m[w] = anc[p][w];
        next = up[p];
      }
      __syncthreads();
      if (j < nodes) {
        for (int w = 0; w < kWords; ++w) anc[j][w] |= m[w];
        up[j] = next;
      }
      __syncthreads();
    }
  }
};

}  // namespace tfx
