// Checks of arguments that the entry points of tf_spec.h and tf_qcache.h share.
#pragma once

#include <cmath>
#include <cstdint>
#include <limits>

#include "spec.h"

namespace tfx {

inline constexpr int64_t kMaxRows = int64_t{1} << 24;  // batch * nodes * heads of one call

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool eights(int64_t a, int64_t b, int64_t c) { return ((a | b | c) & 7) == 0; }

// Whether two arrays of 32-bit numbers share any.
inline bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uint64_t>(nb) * 4 && y < x + static_cast<uint64_t>(na) * 4;
}

// Whether the factor of a score is a number in fp32 (false for NaN).
inline bool fp32_scale(double scale) {
  return std::fabs(scale) <= std::numeric_limits<float>::max() && std::isfinite(static_cast<float>(scale) * kLog2e);
}

inline tf_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TF_OK : record_cuda_error(e, what); }

}  // namespace tfx
