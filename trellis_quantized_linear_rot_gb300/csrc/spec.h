// Internal types and launchers of the operators declared in tf_spec.h.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "per_device.h"
#include "tf_spec.h"

namespace tfx {

constexpr int kErrWait = 1;   // device error bits: a bounded wait gave up,
constexpr int kErrIndex = 2;  // an index outside its array was skipped

// Division of numbers below 2^31 by a divisor known on the host, by Granlund
// and Montgomery's multiplier and shift: two instructions on the device
// instead of about twenty.
struct FastDiv {
  uint32_t mul = 0, shift = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
#endif
};

// The fields of tf_kv_cache the kernels read, without the array pointers.
struct CacheView {
  int64_t stride_layer, stride_page, stride_token, stride_head;
  const int32_t* page_table;
  const int32_t* lengths;
  int64_t stride_table;
  int layers, pages, page_size, kv_heads, head_dim, batch, table_width;
  FastDiv by_page;
  int* err;
};

struct AttendArgs {
  CacheView c;
  const void* k;
  const void* v;
  const void* q;
  int64_t q_seq, q_node, q_head;
  const int32_t* parents;
  int64_t stride_parents;
  void* out;
  float* lse;
  int nodes, heads, group;
  float scale;
  float* partials;
  int* counters;
  int num_sms;
  int join_later;   // the parts are joined by a launch of their own
};

// Scores are scaled by scale * kLog2e, in fp32.
constexpr float kLog2e = 1.4426950408889634f;

// Blocks of an attention launch for each SM.
constexpr int kBlocksPerSm = 2;

// A workspace begins with counters for the most blocks that any attention
// kernel launches, so that the parts of a call over a 16-bit cache never lie
// where the counters of one over a quantised cache are.
constexpr int kMostBlocksPerSm = 4;
static_assert(kBlocksPerSm <= kMostBlocksPerSm, "counters for each block");
inline size_t attend_counter_bytes(int num_sms) {
  return (2 * static_cast<size_t>(kMostBlocksPerSm) * num_sms * sizeof(int) + 255) & ~static_cast<size_t>(255);
}

struct AttendWorkspace {
  size_t partials_at, bytes;
};
AttendWorkspace attend_workspace(int nodes, int heads, int kv_heads, int head_dim, int num_sms);

struct VerifyArgs {
  const void* logits;
  const void* draft;
  int64_t seq, node, draft_seq, draft_node;
  const int32_t* tokens;
  const int32_t* parents;
  int64_t stride_parents;
  const float* u_accept;
  const float* u_sample;
  float inv_temp;
  int greedy;
  int batch, nodes, vocab;
  int32_t* counts;
  int32_t* path;
  int32_t* out_tokens;
  float* logprobs;
  int* work;   // [3][batch * nodes] decisions, [batch] counters, all zero between calls
  int* err;
  int num_sms;
};
size_t verify_workspace_bytes(int batch, int nodes, int num_sms);

// Launches with programmatic stream serialisation: the kernel may be set up
// while the one before it still runs. Every thread of every kernel launched
// this way waits for that one (chain()) before it returns, and before it
// touches anything that one may write, or writes anything that one may read.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream,
                           A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
}

cudaError_t launch_kv_write(const CacheView& c, void* k, void* v, const void* k_new, const void* v_new,
                            int64_t seq, int64_t node, int64_t head, int nodes, cudaStream_t s);
cudaError_t launch_kv_keep(const CacheView& c, void* k, void* v, const int32_t* path, const int32_t* counts,
                           int nodes, int32_t* new_lengths, cudaStream_t s);
cudaError_t launch_tree_attention(const AttendArgs& a, int dtype, int device, cudaStream_t s);
cudaError_t launch_verify_draft(const VerifyArgs& a, int dtype, cudaStream_t s);

}  // namespace tfx
