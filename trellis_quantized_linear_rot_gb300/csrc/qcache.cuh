// Device helpers shared by the kernels of the quantised cache.
#pragma once

#include "qcache.h"
#include "spec.cuh"

namespace tfx {

// Where slot `slot` of sequence `b` lies: its page and row; false where it
// lies past the table or its page outside the pool (recorded).
struct Place {
  int page, row;
};
__device__ __forceinline__ bool place_of(const CacheView& c, int b, int64_t slot, Place* p) {
  if (slot < 0 || slot >= slot_capacity(c)) {
    record_index_error(c.err);
    return false;
  }
  const int t = c.by_page(static_cast<int>(slot));
  p->page = c.page_table[b * c.stride_table + t];
  p->row = static_cast<int>(slot) - t * c.page_size;
  if (p->page < 0 || p->page >= c.pages) {
    record_index_error(c.err);
    return false;
  }
  return true;
}
__device__ __forceinline__ int64_t codes_at(const CacheView& c, const Place& p) {
  return p.page * c.stride_page + p.row * c.stride_token;
}
__device__ __forceinline__ int64_t scales_at(const QView& q, const Place& p) {
  return p.page * q.scale_page + p.row * q.scale_token;
}

// The factors of key (low half) and value of a word.
__device__ __forceinline__ float key_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float value_scale(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight 16-bit elements as fp32 and back.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f32(t[i]);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  alignas(16) T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(x[i]);
  return *reinterpret_cast<const uint4*>(t);
}

}  // namespace tfx
